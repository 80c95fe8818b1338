"""Routing of any number of tokens against exact logits, and grouping of slots."""

import math

import pytest
import torch

import prompt64 as p64

pytestmark = pytest.mark.gpu
H, E, K = 2816, 128, 8


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


def inputs(T, seed, strong=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda")
    if strong:
        x[:, 7::401] *= 12
    w = (torch.randn(E, H, generator=g, device="cuda") * 0.02).bfloat16()
    return x.bfloat16(), w, torch.randn(E, generator=g, device="cuda")


def check(fgm, x, w, b, ws=None, status=0):
    T = x.shape[0]
    ws = fgm.Workspace("cuda", nbytes=fgm.moe_route_workspace_bytes(T)) if ws is None else ws
    r = fgm.moe_route(w, x, b, ws=ws)
    assert ws.status() == status
    ids, wt, top = p64.route(w, x, b)
    assert torch.equal(r.ids.long(), ids)
    # a logit is off by 2^-18 |x| |w| and 2^-23 of itself, a weight by twice that of itself, and by the softmax's own roundings
    dz = 2.0 ** -18 * x.double().norm(dim=1, keepdim=True) * w.double().norm(dim=1).max() + 2.0 ** -23 * torch.where(top.isfinite(), top.abs(), 0.0).amax(dim=1, keepdim=True)
    p64.within(r.weights, wt, wt * (torch.exp(4 * dz) - 1 + 2.0 ** -19))
    offsets, order = p64.group(ids, E)
    assert r.offsets.tolist() == offsets and r.order.tolist() == order
    return r


@pytest.mark.parametrize("T", [1, 2, 5, 8, 31, 127, 128, 129, 257, 1000, 1664, 1665, 5003])
@pytest.mark.parametrize("bias", [False, True])
def test_tokens(fgm, T, bias):
    x, w, b = inputs(T, T)
    check(fgm, x, w, b if bias else None)


def test_no_near_pair_goes_by_fp32(fgm):
    """Routers whose rows differ by one bf16 step in one place: logits 2^-14 and less apart."""
    x, w, _ = inputs(64, 3)
    for e in range(1, E):
        if e % 4:
            w[e] = w[e - e % 4]
            at = (e * 37) % H
            w[e, at] = w[e, at] * (1 + 2.0 ** -7 * (e % 4))
    check(fgm, x, w, None)


def test_equal_rows_take_the_lower_index(fgm):
    x, w, b = inputs(40, 4)
    w[1::2] = w[::2]
    b[1::2] = b[::2]
    check(fgm, x, w, b)
    check(fgm, x, w[:1].repeat(E, 1).contiguous(), None)


@pytest.mark.parametrize("T", [7, 2500])
@pytest.mark.parametrize("alike", [3, 9, 33, 40, 65])
def test_many_near_experts(fgm, T, alike):
    """Tokens side by side of which some have none, some few and some many logits that are near."""
    x, w, b = inputs(T, 10 + alike)
    w[20:20 + alike] = w[20]
    b[20:20 + alike] = b[20] + torch.arange(alike, device="cuda") % 3 * 2.0 ** -20
    check(fgm, x, w, b)
    w[21:20 + alike:2, ::401] *= 1 + 2.0 ** -7
    check(fgm, x, w, b)


def test_tokens_of_zeros(fgm):
    x, w, b = inputs(33, 5)
    x[::3] = 0
    check(fgm, x, w, b)
    assert check(fgm, torch.zeros_like(x), w, None).ids.tolist() == [list(range(8))] * 33


@pytest.mark.parametrize("mask", [-math.inf, torch.finfo(torch.float32).min, -1e30])
@pytest.mark.parametrize("left", [128, 20, 8, 3, 0])
def test_masked_experts(fgm, mask, left):
    x, w, b = inputs(70, 6)
    b[left:] = mask
    b = b[torch.randperm(E, generator=torch.Generator().manual_seed(1)).cuda()].contiguous()
    if left == 0 and mask == -math.inf:            # nothing to choose: the first eight, evenly
        r = fgm.moe_route(w, x, b)
        assert r.ids.tolist() == [list(range(8))] * 70 and (r.weights == 0.125).all()
    else:
        check(fgm, x, w, b)


def test_not_a_number(fgm):
    x, w, b = inputs(20, 7)
    x[3, 100] = math.nan
    b[5] = math.nan
    T = x.shape[0]
    ws = fgm.Workspace("cuda", nbytes=fgm.moe_route_workspace_bytes(T))
    r = fgm.moe_route(w, x, b, ws=ws)
    assert ws.status() == fgm.STATUS_NONFINITE_LOGITS
    ids, wt, _ = p64.route(w, x, b)
    keep = [t for t in range(T) if t != 3]
    assert torch.equal(r.ids.long()[keep], ids[keep]) and not (r.ids == 5)[keep].any()
    assert r.ids[3].tolist() == list(range(8)) and (r.weights[3] == 0.125).all()


def test_rows_apart(fgm):
    x, w, b = inputs(300, 8)
    wide = torch.full((300, H + 24), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + H] = x
    a, c = fgm.moe_route(w, wide[:, 8:8 + H], b), fgm.moe_route(w, x, b)
    for i, j in zip(a, c):
        assert torch.equal(i, j)


def test_sizes_of_values(fgm):
    x, w, b = inputs(50, 9)
    for e in (-30, 20):
        check(fgm, (x.float() * 2.0 ** e).bfloat16(), w, None)
    check(fgm, x, w, b * 1e4)


@pytest.mark.parametrize("n,E_", [(1, 1), (7, 3), (40, 128), (1024, 128), (1025, 128), (5000, 1), (5000, 1024), (70001, 60), (300007, 128)])
def test_groups(fgm, n, E_):
    g = torch.Generator().manual_seed(n)
    ids = torch.randint(-2, E_ + 2, (n,), generator=g, dtype=torch.int32)
    ids[ids == E_ + 1] = torch.iinfo(torch.int32).max
    ids[ids == -2] = torch.iinfo(torch.int32).min
    order = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    off, order = fgm.moe_group(ids.cuda(), E_, order=order)
    want, slots = p64.group(ids, E_)
    assert off.tolist() == want
    assert order.tolist() == slots + [-7] * (n - len(slots))


def test_groups_of_nothing_and_of_one(fgm):
    off, order = fgm.moe_group(torch.full((600,), -1, dtype=torch.int32, device="cuda"), 5, order=torch.full((600,), 3, dtype=torch.int32, device="cuda"))
    assert off.tolist() == [0] * 6 and (order == 3).all()
    off, order = fgm.moe_group(torch.full((3000,), 4, dtype=torch.int32, device="cuda"), 5)
    assert off.tolist() == [0] * 5 + [3000] and order.tolist() == list(range(3000))


@pytest.mark.parametrize("T", [4097, 32769, 40961])
def test_long_prompts_grouped_again(fgm, T):
    """Chunks of 1,024 slots and of more, one workspace for other tokens, in a replayed graph, too."""
    x, w, b = inputs(T, T)
    ws = fgm.Workspace("cuda", nbytes=fgm.moe_route_workspace_bytes(T))
    r = fgm.moe_route(w, x, b, ws=ws)
    ids = r.ids.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fgm.moe_route(w, x, b, out=r, ws=ws)
    for _ in range(3):
        order = torch.sort(r.ids.flatten(), stable=True).indices
        assert torch.equal(r.order.long(), order)
        assert r.offsets.tolist() == [0] + torch.bincount(r.ids.flatten(), minlength=E).cumsum(0).tolist()
        x.copy_(x.flip(0))
        graph.replay()
        ids = ids.flip(0)
        assert torch.equal(r.ids, ids)
    assert ws.status() == 0


def test_binding_refusals(fgm):
    x, w, b = inputs(4, 1)
    for call in (lambda: fgm.moe_route(w, x.float()), lambda: fgm.moe_route(w, x[:, :2800]), lambda: fgm.moe_route(w[:64], x),
                 lambda: fgm.moe_route(w, x, b[:5]), lambda: fgm.moe_route(w, x.t()), lambda: fgm.moe_route(w, x[:0]),
                 lambda: fgm.moe_group(torch.zeros(4, device="cuda"), 3), lambda: fgm.moe_group(torch.zeros(4, dtype=torch.int32, device="cuda"), 0),
                 lambda: fgm.moe_route(w, x, ws=fgm.Workspace("cuda", nbytes=0))):
        with pytest.raises(fgm.FgmError):
            call()
