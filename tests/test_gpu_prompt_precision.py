"""What include/fgm.h promises of the precision of products on E4M3 weights and of the experts,
with its absolute floors, where activations and scales lie far apart."""

import pytest
import torch

import prompt64 as p64
from test_gpu_moe_experts import H, fgm, layer, run, tokens  # noqa: F401 (fgm, layer: fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("largest", [128, 129, 191, 192, 254, 255])
def test_elements_of_a_row(fgm, largest):
    """Weights of ones on the diagonal give back what a row's elements entered as."""
    n = 512
    v = torch.arange(1, 0x7F80, 7, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    v = v[(v.float() >= 2.0 ** -30 * largest) & (v.float() <= largest)]
    v = torch.cat([v, -v])
    v = torch.nn.functional.pad(v, (0, -len(v) % (n - 1))).view(-1, n - 1)
    x = torch.cat([v, torch.full((len(v), 1), float(largest), dtype=torch.bfloat16, device="cuda")], dim=1)
    x[1::2] *= 2.0 ** -70
    x[2::4] *= 2.0 ** 60
    w = torch.where(torch.eye(n, device="cuda") > 0, 0x38, 0).to(torch.uint8)[None].contiguous()
    out = fgm.grouped_gemm(x, w, None, torch.tensor([0, len(x)], dtype=torch.int32, device="cuda")).double()
    x, top = x.double(), x.double().abs().amax(dim=1, keepdim=True)
    assert torch.equal(torch.where(x.abs() >= 2.0 ** -9 * top, out, 0.0), torch.where(x.abs() >= 2.0 ** -9 * top, x, 0.0))
    assert ((out - x).abs() <= 2.0 ** -17 * top).all()


def experts_bound(L, x, e):
    """One expert's rows in 64 bits and the documented bounds: x's terms, activations as f16 and two terms, the output's
    2^-11 of itself or 2^-19 of the largest activation times the largest scale; sums as in prompt64."""
    g, dg = p64.products(x, p64.e4m3(L["gate_q"][e]), L["gate_s"][e].double(), True)
    u, du = p64.products(x, p64.e4m3(L["up_q"][e]), L["up_s"][e].double(), True)
    a = p64.gelu(g) * u
    da = 1.13 * dg * (u.abs() + du) + p64.gelu(g).abs() * du + (2.0 ** -11 + 2.0 ** -20) * a.abs()
    top = (a.abs() + da).amax(dim=1, keepdim=True)
    da = da + torch.maximum(2.0 ** -9 * (a.abs() + da), 2.0 ** -17 * top)
    w, s = p64.e4m3(L["down_q"][e]), L["down_s"][e].double()
    o = (a @ w.t()) * s
    do = (da @ w.abs().t() + 44 * p64.ADD * ((a.abs() + da) @ w.abs().t())) * s.abs()
    return o, do + torch.maximum(2.0 ** -11 * (o.abs() + do), 2.0 ** -19 * top * s.abs().max())


@pytest.mark.parametrize("step", [1, 2, 3])
def test_down_scales_far_apart(fgm, layer, step):
    """Features whose down scales go down to 2^-45 of their expert's largest."""
    L = dict(layer)
    L["down_s"] = layer["down_s"] * torch.exp2(-step * (torch.arange(H, device="cuda") % 16).float())
    x, ids, w = tokens(50, 30 + step)
    ids[:], w[:] = -1, 0
    ids[:, 3], w[:, 3] = 17, 1
    y = run(fgm, L, x, ids, w, False)
    want, err = experts_bound(L, x, 17)
    p64.within(y, want, p64.rounded(want, err, torch.bfloat16))


def test_activations_far_apart(fgm, layer):
    """Gate scales that leave a few activations far above the others."""
    L = dict(layer)
    L["up_s"] = layer["up_s"] * torch.exp2(-(torch.arange(704, device="cuda") % 24).float())
    x, ids, w = tokens(50, 40)
    ids[:], w[:] = -1, 0
    ids[:, 0], w[:, 0] = 90, 1
    y = run(fgm, L, x, ids, w, False)
    want, err = experts_bound(L, x, 90)
    p64.within(y, want, p64.rounded(want, err, torch.bfloat16))
