"""Workspaces and layers on another device than a call's tensors are refused: stand-ins
for tensors of a second GPU, no GPU needed."""

from types import SimpleNamespace

import pytest
import torch

import fine_grained_moe_gb300 as fgm

FIRST, SECOND = torch.device("cuda", 0), torch.device("cuda", 1)


class Stand:
    """As much of a tensor as the checks of a layer look at."""

    is_cuda = True

    def __init__(self, shape, dtype, device=FIRST):
        self.shape, self.dtype, self.device = shape, dtype, device

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


def layer(**other):
    F, H, E, N = fgm.FFN, fgm.HIDDEN, fgm.EXPERTS, fgm.N_EXPERTS
    shapes = dict(router_w=((E, H), torch.bfloat16), router_b=((E,), torch.float32), gate_q=((N, F, H), torch.uint8),
                  gate_s=((N, F), torch.float32), up_q=((N, F, H), torch.uint8), up_s=((N, F), torch.float32),
                  down_q=((N, H, F), torch.uint8), down_s=((N, H), torch.float32))
    return {n: Stand(s, t, other.get(n, FIRST)) for n, (s, t) in shapes.items()}


@pytest.mark.parametrize("name", [n for n in layer() if not n.startswith("router")])
def test_layers_elsewhere(name):
    assert fgm._layer_on(layer(), FIRST).gate_q == 4096
    with pytest.raises(fgm.FgmError, match=name):
        fgm._layer_on(layer(**{name: SECOND}), FIRST)
    with pytest.raises(fgm.FgmError):
        fgm._layer_on(layer(), SECOND)


def test_a_layer_without_a_bias():
    assert fgm._layer_on(dict(layer(), router_b=None), FIRST).down_s == 4096


def test_workspaces_elsewhere():
    ws = SimpleNamespace(t=SimpleNamespace(device=FIRST))
    assert fgm._space(ws, FIRST) is ws
    with pytest.raises(fgm.FgmError, match="workspace"):
        fgm._space(ws, SECOND)
