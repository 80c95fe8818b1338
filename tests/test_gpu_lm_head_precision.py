"""What fgm_lm_head_logprobs on more than 8 rows does with the logits that its
first pass gets only to the tensor pipe's truncation: the largest are computed
again in fp32, at every temperature.

Errors. A logit computed again is a sum of 88 products a lane in two chains and 6
additions over the lanes, all in fp32: off by at most dz = (44 + 6) 2^-24 S, S the
largest sum |h e|. Outputs are differences of two such logits over T, and sums of
fp32 terms: |err| <= 2 dz / T + 2^-18 + 2^-22 |want|.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
H = 2816
DEV = "cuda"


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


def planted(N, V, sign, seed):
    """Rows with five words about 4 apart over a floor below them; sign < 0: every logit is negative."""
    g = torch.Generator().manual_seed(seed)
    emb = torch.randn(V, H, generator=g) * 0.02
    h = torch.randn(N, H, generator=g) * 0.1
    pick = torch.stack([torch.randperm(V, generator=g)[:5] for _ in range(N)])
    for i in range(5):
        h += (22.0 - 4.0 * i) / 1.126 * emb[pick[:, i]]
    if sign < 0:
        emb += 0.02
        h -= 0.6
    emb, h = emb.bfloat16().to(DEV), h.bfloat16().to(DEV)
    z = h.double() @ emb.double().t()
    S = float((h.double().abs() @ emb.double().abs().t()).max())
    return emb, h, z, S


@pytest.mark.parametrize("T", [2.95e-39, 1e-30, 1e-9, 1e-6, 1e-3, 0.05, 1.0])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("N,V,k", [(9, 5003, 4), (300, 20011, 6), (300, 20011, 12)])
def test_temperatures(fgm, N, V, k, sign, T):
    emb, h, z, S = planted(N, V, sign, N + V)
    dz = 50 * 2.0 ** -24 * S
    T32 = float(np.float32(T))
    top = torch.sort(z, dim=1, descending=True)
    gap = (top.values[:, :4] - top.values[:, 1:5]).min()
    assert float(gap) > 0.2 and (float(top.values[:, 0].max()) < 0) == (sign < 0)
    tokens = top.indices[:, 0].to(torch.int32)
    tokens[::3] = top.indices[::3, 2].to(torch.int32)
    ws = fgm.Workspace("cuda", nbytes=fgm.lm_head_logprobs_workspace_bytes(N, V, k))
    r = fgm.lm_head_logprobs(emb, h, tokens, k=k, T=T, ws=ws)
    assert ws.status() == 0
    x = (z - top.values[:, :1]) / T32
    lnl = torch.logsumexp(x, dim=1, keepdim=True)
    lp = x - lnl
    # what the words behind the recomputed ones add is off by their logits' truncation, 176 ulps of them, over T
    rest = top.values[:, 12:]
    share = torch.exp((rest - top.values[:, :1]) / T32).sum(dim=1, keepdim=True)
    far = share * (1 - torch.exp(torch.tensor(-min(700.0, 176 * 2.0 ** -23 * float(rest.abs().max()) / T32), dtype=torch.float64, device="cuda")))
    lowest = 3.4028234e38

    def near(got, want, what, extra=0.0):
        got = got.double()
        tol = 2 * dz / T32 + 2.0 ** -18 + 2.0 ** -22 * want.abs() + 2 * far[:, :1].expand(want.shape) + extra
        ok = (got - want).abs() <= tol
        # (beyond fp32: -inf; within the bound of its limit either may stand)
        ok |= (got == -float("inf")) & (want <= -(lowest - tol))
        assert ok.all(), (what, got[~ok][:4].tolist(), want[~ok][:4].tolist())

    near(r.logp[:, None], lp.gather(1, tokens.long()[:, None]), "logp")
    near(r.top_logp[:, :4], lp.gather(1, top.indices[:, :4]), "top_logp")
    assert torch.equal(r.top_ids[:, :4].long(), top.indices[:, :4])
    # the largest stands gap / T above the next: its own bound
    best = r.top_logp[:, 0].double()
    second = float(gap) - 2 * dz
    assert (best <= 2.0 ** -18).all()
    assert (best >= -(V * np.exp(-min(700.0, second / T32)) + 2.0 ** -18)).all()
    p = torch.exp(lp)
    ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(dim=1)
    tail = V * np.exp(-min(700.0, second / T32)) * (1 + min(700.0, second / T32))      # the entropy that is there at most
    et = (2 * dz / T32 + 2.0 ** -18 + 2 * far[:, 0]) * (1 + ent + np.log(V))
    e = r.entropy.double()
    assert torch.isfinite(e).all()
    assert (((e - ent).abs() <= et) | (e.abs() <= tail + 2.0 ** -18)).all()


@pytest.mark.parametrize("T", [1.0, 0.01])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("N", [9, 130])
def test_products_that_the_first_pass_drops(fgm, N, sign, T):
    """Word 7's logit is 16 and 2,815 products of 2^-24, 16 of which together are
    half an ulp of 16; word 300's is 16 alone, so the two differ by 2815 2^-24 =
    1.68e-4. In the fp32 sum the chain with the 16 drops at most 43 of them and 6
    additions round by half an ulp of 16, 2^-20 each: dz = 43 2^-24 + 6 2^-20 =
    8.3e-6 (word 300: exact)."""
    V = 600
    emb = torch.zeros(V, H)
    if sign < 0:
        emb[:, 0] = -8.0
    emb[7, 0] = emb[300, 0] = 4.0 * sign
    emb[7, 1:] = 2.0 ** -12 * sign
    h = torch.full((N, H), 2.0 ** -12)
    h[:, 0] = 4.0
    emb, h = emb.bfloat16().cuda(), h.bfloat16().cuda()
    z = (h.double() @ emb.double().t())
    diff = float(z[0, 7] - z[0, 300])
    assert abs(abs(diff) - 2815 * 2.0 ** -24) < 1e-12
    first, second = (7, 300) if sign > 0 else (300, 7)
    tokens = torch.full((N,), 7, dtype=torch.int32, device="cuda")
    ws = fgm.Workspace("cuda", nbytes=fgm.lm_head_logprobs_workspace_bytes(N, V, 2))
    r = fgm.lm_head_logprobs(emb, h, tokens, k=2, T=T, ws=ws)
    assert ws.status() == 0
    T32 = float(np.float32(T))
    lp = torch.log_softmax(z / T32, dim=1)
    ent = -(torch.exp(lp) * torch.where(torch.isfinite(lp), lp, torch.zeros_like(lp))).sum(dim=1)
    tol = (43 * 2.0 ** -24 + 6 * 2.0 ** -20) / T32 + 2.0 ** -18 + 2.0 ** -22
    assert (r.top_ids.long() == torch.tensor([first, second], device="cuda")).all()
    want = lp[:, [first, second]]
    assert ((r.top_logp.double() - want).abs() <= tol).all(), ((r.top_logp.double() - want).abs().max(), tol)
    assert ((r.logp.double() - lp[:, 7]).abs() <= tol).all()
    assert ((r.entropy.double() - ent).abs() <= 2 * tol).all(), ((r.entropy.double() - ent).abs().max(), tol)


def test_rows_alike_on_either_side_of_eight(fgm):
    """The same rows among 5 and among 40, at a low temperature: both are within their bounds of the same numbers."""
    emb, h, z, S = planted(40, 9001, 1, 5)
    dz = 50 * 2.0 ** -24 * S + 2816 * 2.0 ** -23 * 13
    tokens = torch.sort(z, dim=1, descending=True).indices[:, 1].to(torch.int32).contiguous()
    for T in (1e-6, 0.02):
        a = fgm.lm_head_logprobs(emb, h, tokens, k=3, T=T)
        b = fgm.lm_head_logprobs(emb, h[:5].contiguous(), tokens[:5].contiguous(), k=3, T=T)
        assert torch.equal(a.top_ids[:5], b.top_ids)
        assert torch.isfinite(a.logp).all() and torch.isfinite(a.top_logp).all() and torch.isfinite(a.entropy).all()
        assert ((a.logp[:5] - b.logp).abs() <= 4 * dz / T + 2.0 ** -17).all()
        assert ((a.entropy[:5] - b.entropy).abs() <= 2.0 ** -17).all()
