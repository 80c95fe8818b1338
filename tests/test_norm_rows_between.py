"""Block norms whose gate or gains of one row lie between the rows of an output: allowed, as
no byte is shared. On the CPU what passes the checks is refused for want of a GPU alone."""

import ctypes

import pytest
import torch

import fine_grained_moe_gb300 as fgm
import prompt64 as p64
from test_prompt_abi import AT, block, lib  # noqa: F401 (lib: the fixture)

WIDE = dict(h=AT, y=AT + 128, h_out=AT + 256, xn=AT + 5120, h_stride=256, y_stride=256, h_out_stride=256, gain_type=1, pre_gain=None)


def one(at):
    """A gate of one row for all."""
    return dict(WIDE, gate=AT + at, gate_row_stride=0, post_gain=None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="host addresses must not reach a GPU")
@pytest.mark.parametrize("good", [
    one(384), one(512 + 384), one(3 * 512 + 384), dict(one(384), post_gain=AT + 512 + 384), dict(one(384), pre_gain=AT + 1024 + 384),
    dict(one(384), N=1), dict(one(384), xn=AT + 1920, xn_stride=256, h_out=None)])
def test_between(lib, good):
    assert lib.fgm_block_norm(ctypes.byref(block(**good)), None) in (-3, -4), lib.fgm_last_error()


@pytest.mark.parametrize("bad", [one(256), one(258), one(382), one(256 + 512 - 126), one(1024 + 260), dict(one(384), post_gain=AT + 512 + 300),
                                 dict(one(384), pre_gain=AT + 1024 + 200), dict(one(256), N=1)])
def test_shared_bytes(lib, bad):
    assert lib.fgm_block_norm(ctypes.byref(block(**bad)), None) == -1 and b"overlaps" in lib.fgm_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 130])
def test_a_gate_and_gains_between_rows(D):
    g = torch.Generator(device="cuda").manual_seed(D)
    wide = torch.randn(300, 4 * D, generator=g, device="cuda").bfloat16()
    h, y, o, rest = (wide[:, i * D:(i + 1) * D] for i in range(4))
    gate, post, pre = rest[0], rest[7], rest[299]
    keep = wide.clone()
    want, dw, wn, dn = p64.block(h.clone(), y.clone(), post.clone(), gate.clone(), pre.clone(), True, 1.0, 1.0, 0.0, 1e-6)
    out, xn = fgm.block_norm(h, y, post_gain=post, gate=gate, pre_gain=pre, h_out=o)
    p64.within(out, want, p64.rounded(want, dw, torch.bfloat16))
    p64.within(xn, wn, p64.rounded(wn, dn, torch.bfloat16))
    keep[:, 2 * D:3 * D] = o
    assert torch.equal(keep, wide)
