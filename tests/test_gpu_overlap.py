"""Launches that overlap the ones before them: a run of appends and attentions with
nothing between them, in one graph, gives the bits of the same calls one at a time."""

import pytest
import torch

from test_gpu_kv_cache import random_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


def test_appends_and_attentions_back_to_back(fgm):
    """Every append makes its block's scales grow, so that an attention that read
    older ones would be off by factors."""
    H, G, M, D, steps = 4, 2, 1, 128, 40
    g = torch.Generator().manual_seed(4)
    q = torch.randn(1, M, H * G, D, generator=g).bfloat16().cuda()
    grow = torch.pow(1.5, torch.arange(steps).float())[:, None, None, None, None] * 0.01
    k, v = ((torch.randn(steps, 1, 1, H, D, generator=g) * grow).bfloat16().cuda() for _ in range(2))
    lens = [torch.tensor([130 + i], dtype=torch.int32, device="cuda") for i in range(steps)]
    tab = torch.tensor([[3, 0, 2]], dtype=torch.int32, device="cuda")
    ws = fgm.Workspace("cuda", nbytes=fgm.attn_workspace_bytes(1, M, H * G, H, D))

    def run(c, outs, wait):
        for i in range(steps):
            fgm.kv_append(c, k[i], v[i], lens[i], block_table=tab, ws=ws)
            if wait:
                torch.cuda.synchronize()
            fgm.attn_fwd(c, q, lens[i], 0.09, block_table=tab, out=outs[i], ws=ws)
            if wait:
                torch.cuda.synchronize()

    a, b = random_cache(fgm, 4, H, D, seed=1), random_cache(fgm, 4, H, D, seed=1)
    start = [t.clone() for t in (b.k_q, b.v_q, b.k_s, b.v_s)]
    apart = torch.zeros(steps, 1, M, H * G, D, dtype=torch.bfloat16, device="cuda")
    close = torch.zeros_like(apart)
    run(a, apart, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b, close, False)
    for _ in range(5):
        for t, s in zip((b.k_q, b.v_q, b.k_s, b.v_s), start):
            t.copy_(s)
        close.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(close, apart)
        for name in ("k_q", "v_q", "k_s", "v_s"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
    assert ws.status() == 0
