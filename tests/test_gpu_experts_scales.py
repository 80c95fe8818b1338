"""Experts whose down scales lie near the end of fp32's range, with activations as small."""

import pytest
import torch

from test_gpu_moe_experts import check, fgm, layer, tokens  # noqa: F401 (fgm, layer: fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("down", [100, 118, 124])
def test_large_down_scales(fgm, layer, down):
    """Outputs of ordinary size: activations 2^-100 times, down scales up to 2^124."""
    L = dict(layer)
    for n in ("gate_s", "up_s"):
        L[n] = layer[n] * 2.0 ** -50
    top = layer["down_s"].double().amax()
    L["down_s"] = (layer["down_s"].double() * (2.0 ** down / top)).float()
    x, ids, w = tokens(30, down)
    y = check(fgm, L, x, ids, w)
    assert y.isfinite().all()


def test_small_down_scales(fgm, layer):
    L = dict(layer)
    for n in ("gate_s", "up_s"):
        L[n] = layer[n] * 2.0 ** 45
    L["down_s"] = layer["down_s"] * 2.0 ** -100
    x, ids, w = tokens(30, 3)
    check(fgm, L, x, ids, w)
