"""Routing by exact logits over the range of bf16: rows whose squares pass fp32's range
at either end, and routers with rows that are not finite, or far from the others."""

import math

import pytest
import torch

import prompt64 as p64
from test_gpu_route import E, H, fgm, inputs  # noqa: F401 (fgm: the fixture)

pytestmark = pytest.mark.gpu


def near_rows(w):
    """Rows in fours that differ by single bf16 steps in one place."""
    for e in range(1, E):
        if e % 4:
            w[e] = w[e - e % 4]
            at = (e * 37) % H
            w[e, at] = w[e, at] * (1 + 2.0 ** -7 * (e % 4))
    return w


def check(fgm, x, w, b, status=(0,), weights=True):
    T = x.shape[0]
    ws = fgm.Workspace("cuda", nbytes=fgm.moe_route_workspace_bytes(T))
    r = fgm.moe_route(w, x, b, ws=ws)
    assert ws.status() in status
    ids, wt, _ = p64.route(w, x, b)
    assert torch.equal(r.ids.long(), ids), int((r.ids.long() != ids).any(dim=1).sum())
    offsets, order = p64.group(ids, E)
    assert r.offsets.tolist() == offsets and r.order.tolist() == order
    if weights:                                    # (logits far below 1: all alike, to the softmax's own roundings)
        p64.within(r.weights, wt, wt * 2.0 ** -19)
    return r


@pytest.mark.parametrize("T", [5, 300, 9729])
@pytest.mark.parametrize("ex,ew", [(-90, 0), (-120, 0), (-75, 0), (-60, 0), (-46, -46), (-60, -60), (0, -70), (0, -100), (30, -80)])
def test_small_rows(fgm, T, ex, ew):
    x, w, _ = inputs(T, 3)
    x = (x.float() * 2.0 ** ex).bfloat16()
    w = near_rows((w.float() * 2.0 ** ew).bfloat16())
    x[1::7] = 0                                    # (and tokens of zeros among them: the first eight)
    r = check(fgm, x, w, None)
    assert (r.ids[1::7] == torch.arange(8, device="cuda")).all()


@pytest.mark.parametrize("T", [5, 300, 9729])
@pytest.mark.parametrize("ex,ew", [(70, 0), (100, 0), (60, 40), (0, 70), (0, 100), (110, -60), (-60, 110)])
def test_large_rows(fgm, T, ex, ew):
    x, w, _ = inputs(T, 4)
    x = (x.float() * 2.0 ** ex).bfloat16()
    w = near_rows((w.float() * 2.0 ** ew).bfloat16())
    check(fgm, x, w, None, weights=False)


def test_rows_of_all_sizes_side_by_side(fgm):
    x, w, b = inputs(600, 5)
    w = near_rows(w)
    x = (x.float() * torch.exp2(torch.arange(600, device="cuda") % 200 - 110.0)[:, None]).bfloat16()
    check(fgm, x, w, None, weights=False)


@pytest.mark.parametrize("T", [40, 9729])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_masked_experts_that_are_not_finite(fgm, T, value):
    """A row of the router that holds no numbers, masked by its bias, hides no near pair of the others."""
    x, w, b = inputs(T, 6)
    w = near_rows(w)
    b[:] = 0
    w[7, 5], w[50, 2000:] = value, value
    b[7] = b[50] = -math.inf
    r = check(fgm, x, w, b, status=(fgm.STATUS_NONFINITE_LOGITS, 0))
    assert not ((r.ids == 7) | (r.ids == 50)).any()


@pytest.mark.parametrize("T", [40, 9729])
def test_a_masked_expert_far_larger_than_the_others(fgm, T):
    x, w, b = inputs(T, 7)
    w = near_rows(w)
    b[:] = 0
    w[9] = 2.0 ** 70
    b[9] = -math.inf
    check(fgm, x, w, b)


def test_rows_not_finite_among_others(fgm):
    x, w, _ = inputs(200, 8)
    w = near_rows(w)
    x[4, 9], x[77, 2815] = math.nan, math.nan
    ws = fgm.Workspace("cuda", nbytes=fgm.moe_route_workspace_bytes(200))
    r = fgm.moe_route(w, x, None, ws=ws)
    assert ws.status() == fgm.STATUS_NONFINITE_LOGITS
    ids = p64.route(w, x, None)[0]
    assert torch.equal(r.ids.long(), ids)
    assert (r.weights[[4, 77]] == 0.125).all()


def test_routers_of_zeros(fgm):
    x, w, b = inputs(70, 9)
    assert (check(fgm, x, torch.zeros_like(w), None).ids == torch.arange(8, device="cuda")).all()
    r = fgm.moe_route(torch.zeros_like(w), x, b)
    assert torch.equal(r.ids.long(), torch.sort(b, descending=True, stable=True).indices[:8].expand(70, 8))


@pytest.mark.parametrize("T", [9, 9729])
def test_logits_of_plus_infinity(fgm, T):
    """First in order, lower indices first; without a distribution, as in 64 bits."""
    x, w, b = inputs(T, 10)
    w = near_rows(w)
    b[:] = 0
    b[90] = b[33] = math.inf
    ids, wt, _ = p64.route(w, x, b)
    r = fgm.moe_route(w, x, b)
    assert torch.equal(r.ids.long(), ids) and (r.ids[:, :2] == torch.tensor([33, 90], device="cuda")).all()
    assert r.weights.isnan().all() and wt.isnan().all()
