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


def test_streams_at_once(fgm):
    """Three streams with a workspace each run every operator at the same time; the
    bits are those of the calls one after another."""
    def job(seed):
        g = torch.Generator().manual_seed(seed)
        H, G, M, D = 2, 4, 5, 64 << (seed % 3)
        V, N = 9001, (3, 20, 300)[seed % 3]
        q = torch.randn(2, M, H * G, D, generator=g).bfloat16().cuda()
        k, v = (torch.randn(2, M, H, D, generator=g).bfloat16().cuda() for _ in range(2))
        lens = torch.tensor([900 + seed, 70], dtype=torch.int32, device="cuda")
        tab = torch.randperm(32, generator=g).view(2, 16).to(torch.int32).cuda()
        emb = (torch.randn(V, 2816, generator=g) * 0.02).bfloat16().cuda()
        h = torch.randn(N, 2816, generator=g).bfloat16().cuda()
        z = torch.randn(40, V, generator=g).cuda()
        t = torch.randint(0, V, (300,), generator=g).to(torch.int32).cuda()
        ws = fgm.Workspace("cuda", nbytes=max(fgm.attn_workspace_bytes(2, M, H * G, H, D), fgm.logprobs_workspace_bytes(40, V, 5),
                                              fgm.lm_head_logprobs_workspace_bytes(N, V, 5)))
        cache = random_cache(fgm, 32, H, D, seed=seed)

        def run():
            fgm.kv_append(cache, k, v, lens, block_table=tab, ws=ws)
            out = fgm.attn_fwd(cache, q, lens, D ** -0.5, block_table=tab, ws=ws)
            a = fgm.logprobs(z, t[:40], k=5, ws=ws)
            b = fgm.lm_head_logprobs(emb, h, t[:N], k=5, ws=ws)
            return [out, *a, *b, cache.k_q, cache.v_q, cache.k_s, cache.v_s]
        return run, ws

    jobs = [job(s) for s in range(3)]
    want = [[x.clone() for x in run()] for run, _ in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        got = []
        for s, (run, _) in zip(streams, jobs):
            with torch.cuda.stream(s):
                got.append(run())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
    assert all(ws.status() == 0 for _, ws in jobs)
