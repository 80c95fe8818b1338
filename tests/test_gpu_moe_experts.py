"""A layer's experts on any number of tokens against 64 bits."""

import math

import pytest
import torch

import prompt64 as p64
import synth

pytestmark = pytest.mark.gpu
H = 2816


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def layer():
    return synth.layer(3, device="cuda", s=1.1)


def tokens(T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda")
    x[:, 11::509] *= 15
    z = torch.randn(T, 128, generator=g, device="cuda") - 1.1 * torch.log(torch.arange(128, device="cuda") + 1.0)
    top, ids = torch.topk(z, 8, dim=1)
    return x.bfloat16(), ids.int(), torch.softmax(top, dim=1)


def run(fgm, layer, x, ids, w, shared=True, **kw):
    ws = fgm.Workspace("cuda", nbytes=fgm.moe_experts_workspace_bytes(x.shape[0]))
    y = fgm.moe_experts_fwd(layer, x, ids, w, shared=shared, ws=ws, **kw)
    assert ws.status() == 0
    return y


def check(fgm, layer, x, ids, w, shared=True):
    y = run(fgm, layer, x, ids, w, shared)
    want, err = p64.experts(layer, x, ids, w, shared)
    p64.within(y, want, p64.rounded(want, err, torch.bfloat16))
    return y


@pytest.mark.parametrize("T", [1, 2, 7, 16, 33, 128, 129, 300, 1100])
@pytest.mark.parametrize("shared", [True, False])
def test_tokens(fgm, layer, T, shared):
    x, ids, w = tokens(T, T)
    y = check(fgm, layer, x, ids, w, shared)
    # and not only within the bound of the worst case
    want = p64.experts(layer, x, ids, w, shared)[0]
    assert float((y.double() - want).norm() / want.norm()) < 2.0 ** -8


@pytest.mark.parametrize("T", [4097, 33001])
def test_long_prompts(fgm, layer, T):
    """Chunks of 1,024 slots and of more: the same 300 tokens over and over, each time within the bound."""
    x, ids, w = tokens(300, 12)
    again = torch.arange(T, device="cuda") % 300
    want, err = p64.experts(layer, x, ids, w, True)
    bound = p64.rounded(want, err, torch.bfloat16)
    y = run(fgm, layer, x[again], ids[again], w[again])
    for t in range(0, T, 300):
        n = min(300, T - t)
        p64.within(y[t:t + n], want[:n], bound[:n])


def test_one_expert_for_all(fgm, layer):
    x, ids, w = tokens(700, 5)
    ids[:] = 17                                    # all eight choices the same
    check(fgm, layer, x, ids, w)


def test_places_without_experts(fgm, layer):
    x, ids, w = tokens(150, 6)
    ids[::3] = -1
    ids[1, :4] = 128
    ids[4, 2:] = torch.iinfo(torch.int32).max
    ids[7] = torch.iinfo(torch.int32).min
    w[7] = math.nan                                # (a weight that belongs to no expert is not read)
    real = torch.where((ids < 0) | (ids > 127), -1, ids)
    for shared in (True, False):
        y = run(fgm, layer, x, ids, w, shared)
        want, err = p64.experts(layer, x, real, w, shared)
        p64.within(y, want, p64.rounded(want, err, torch.bfloat16))
    assert (y[::3] == 0).all() and (y[7] == 0).all()
    none = torch.full_like(ids, -1)
    assert (run(fgm, layer, x, none, w, False) == 0).all()


def test_non_finite_tokens_stay_alone(fgm, layer):
    x, ids, w = tokens(40, 7)
    clean = run(fgm, layer, x, ids, w)
    x[5, 9], x[8, 2000] = math.nan, -math.inf
    w[11, 3] = math.nan
    y = run(fgm, layer, x, ids, w)
    assert y[[5, 8, 11]].isnan().all()
    rest = [t for t in range(40) if t not in (5, 8, 11)]
    assert torch.equal(y[rest], clean[rest])


def test_sizes_of_values(fgm, layer):
    x, ids, w = tokens(24, 8)
    x = (x.float() * torch.logspace(-12, 6, 24, device="cuda")[:, None]).bfloat16()
    w = w * torch.logspace(3, -6, 24, device="cuda")[:, None]
    x[3] = 0
    y = check(fgm, layer, x, ids, w)
    assert (y[3] == 0).all()


def test_scales_of_any_size(fgm, layer):
    L = dict(layer)
    g = torch.Generator(device="cuda").manual_seed(9)
    for n in ("gate_s", "up_s", "down_s"):
        L[n] = layer[n] * torch.exp(torch.randn(layer[n].shape, generator=g, device="cuda") * 2)
    L["down_s"][5] = 0
    x, ids, w = tokens(60, 9)
    ids[0, 0] = 5
    check(fgm, L, x, ids, w)


def test_rows_apart_and_their_order(fgm, layer):
    x, ids, w = tokens(90, 10)
    wide = torch.zeros(90, H + 40, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + H] = x
    y = run(fgm, layer, x, ids, w)
    assert torch.equal(run(fgm, layer, wide[:, 16:16 + H], ids, w), y)
    # a token's result does not hang on the others
    few = [3, 50, 89]
    assert torch.equal(run(fgm, layer, x[few].contiguous(), ids[few].contiguous(), w[few].contiguous()), y[few])
    for _ in range(3):
        assert torch.equal(run(fgm, layer, x, ids, w), y)


def test_against_the_verify_steps_layer(fgm, layer):
    """fgm_moe_layer_fwd's tokens, routed and summed by the new calls: both are within their bounds of the same layer."""
    x = synth.hidden_states(4, 5, device="cuda")
    old = fgm.moe_layer_fwd(layer, x)
    r = fgm.moe_route(layer["router_w"], x, layer["router_b"])
    new = run(fgm, layer, x, r.ids, r.weights)
    assert float((old.float() - new.float()).abs().max() / old.float().abs().max()) < 1e-2


def test_places_behind_32_bits(fgm, layer):
    """110,000 tokens: 2.8e9 elements of experts' rows in the workspace."""
    T = 110_000
    x, ids, w = tokens(T, 11)
    y = run(fgm, layer, x, ids, w)
    at = torch.tensor([0, 1, 54_321, T - 2, T - 1], device="cuda")
    want, err = p64.experts(layer, x[at], ids[at], w[at], True)
    p64.within(y[at], want, p64.rounded(want, err, torch.bfloat16))


def test_binding_refusals(fgm, layer):
    x, ids, w = tokens(4, 1)
    for call in (lambda: fgm.moe_experts_fwd(layer, x.float(), ids, w), lambda: fgm.moe_experts_fwd(layer, x, ids.long(), w),
                 lambda: fgm.moe_experts_fwd(layer, x, ids[:, :4], w), lambda: fgm.moe_experts_fwd(layer, x, ids, w.bfloat16()),
                 lambda: fgm.moe_experts_fwd(layer, x, ids, w, y=torch.empty(4, H, device="cuda")),
                 lambda: fgm.moe_experts_fwd(layer, x, ids, w, ws=fgm.Workspace("cuda"))):
        with pytest.raises(fgm.FgmError):
            call()
