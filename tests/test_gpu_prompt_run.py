"""A prompt's way through layers, as a serving loop takes it: norm, routing, experts, norm
and sum, layer after layer, in one captured graph; each operator compared with its plain
64-bit form on the inputs that it had in the run. And several such runs at once."""

import pytest
import torch

import prompt64 as p64
import synth

pytestmark = pytest.mark.gpu
H, EPS = 2816, 1e-6


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def layers():
    return [synth.layer(i, device="cuda", s=1.1) for i in range(2)]


class Prompt:
    """T tokens of a residual stream, fixed buffers, two layers."""

    def __init__(self, fgm, layers, T, seed, h_type=torch.float32):
        self.fgm, self.layers, self.T = fgm, layers, T
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.h0 = torch.randn(T, H, generator=g, device="cuda").to(h_type)
        self.post = [torch.rand(H, generator=g, device="cuda") + 0.5 for _ in layers]
        self.pre = [torch.rand(H, generator=g, device="cuda") + 0.5 for _ in range(len(layers) + 1)]
        self.structs = [fgm.Layer.from_dict(p) for p in layers]
        self.ws = fgm.Workspace("cuda", nbytes=max(fgm.moe_route_workspace_bytes(T), fgm.moe_experts_workspace_bytes(T),
                                                   fgm.grouped_gemm_workspace_bytes(T, 8 * T, 128, 704, H)))

    def run(self):
        """Every tensor that passed between the operators."""
        f, ws, kept = self.fgm, self.ws, []
        h, x = f.block_norm(self.h0, pre_gain=self.pre[0], eps=EPS)
        kept += [h, x]
        for i, (L, p) in enumerate(zip(self.structs, self.layers)):
            r = f.moe_route(p["router_w"], x, p["router_b"], ws=ws)
            gates = f.grouped_gemm(x, p["gate_q"][:128], p["gate_s"][:128], r.offsets, rows=r.order, per=8, ws=ws)
            y = f.moe_experts_fwd(L, x, r.ids, r.weights, ws=ws)
            h, x = f.block_norm(h, y, post_gain=self.post[i], pre_gain=self.pre[i + 1], residual_scale=0.9, eps=EPS)
            kept += [*r, gates, y, h, x]
        return kept


def check_run(p, kept):
    kept = [t.clone() for t in kept]
    h, x = kept[:2]
    for i, L in enumerate(p.layers):
        ids, wt, off, order, gates, y, h1, x1 = kept[2 + 8 * i:10 + 8 * i]
        want_ids, want_w, _ = p64.route(L["router_w"], x, L["router_b"])
        assert torch.equal(ids.long(), want_ids)
        assert float((wt - want_w).abs().max()) < 1e-3
        o, s = p64.group(ids, 128)
        assert off.tolist() == o and order.tolist() == s
        for e in range(128):
            if o[e + 1] > o[e]:
                want, err = p64.products(x[(order[o[e]:o[e + 1]] // 8).long()], p64.e4m3(L["gate_q"][e]), L["gate_s"][e].double(), True)
                p64.within(gates[o[e]:o[e + 1]], want, p64.rounded(want, err, torch.bfloat16))
        want, err = p64.experts(L, x, ids, wt, True)
        p64.within(y, want, p64.rounded(want, err, torch.bfloat16))
        want, dw, wn, dn = p64.block(h, y, p.post[i], None, p.pre[i + 1], True, 0.9, 1.0, 0.0, EPS)
        p64.within(h1, want, p64.rounded(want, dw, h1.dtype))
        p64.within(x1, wn, p64.rounded(wn, dn, torch.bfloat16))
        h, x = h1, x1
    assert p.ws.status() == 0


@pytest.mark.parametrize("T", [1, 37, 600])
def test_layers_in_a_graph(fgm, layers, T):
    p = Prompt(fgm, layers, T, T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = [t.clone() for t in p.run()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = p.run()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(kept, eager):
        assert torch.equal(a, b)
    p.h0.copy_(torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(99), device="cuda") * 3)
    graph.replay()
    torch.cuda.synchronize()
    check_run(p, kept)


def test_graphs_that_share_a_workspace(fgm, layers):
    """One after the other on a stream, in either order, with new inputs between."""
    ps = [Prompt(fgm, layers, T, T) for T in (200, 45)]
    ps[1].ws = ps[0].ws
    graphs, kepts = [], []
    for p in ps:
        p.run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            kepts.append(p.run())
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for p in ps:
            p.h0.normal_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            check_run(ps[i], kepts[i])


def test_streams_at_once(fgm, layers):
    """Three streams with a workspace each; the bits are those of the runs one after another."""
    ps = [Prompt(fgm, layers, T, T, h_type) for T, h_type in ((3, torch.float32), (90, torch.bfloat16), (700, torch.float32))]
    want = [[t.clone() for t in p.run()] for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(10):
        got = []
        for s, p in zip(streams, ps):
            with torch.cuda.stream(s):
                got.append(p.run())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
    assert all(p.ws.status() == 0 for p in ps)


def test_a_stream_of_the_calls_own(fgm, layers):
    p = Prompt(fgm, layers, 20, 5)
    want = [t.clone() for t in p.run()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h, x = fgm.block_norm(p.h0, pre_gain=p.pre[0], eps=EPS, stream=s)
    r = fgm.moe_route(layers[0]["router_w"], x, layers[0]["router_b"], ws=p.ws, stream=s)
    y = fgm.moe_experts_fwd(p.structs[0], x, r.ids, r.weights, ws=p.ws, stream=s)
    off, order = fgm.moe_group(r.ids, 128, ws=p.ws, stream=s)
    gates = fgm.grouped_gemm(x, layers[0]["gate_q"][:128], layers[0]["gate_s"][:128], off, rows=order, per=8, ws=p.ws, stream=s)
    s.synchronize()
    for a, b in zip((h, x, *r, gates, y, off, order), (*want[:8], want[4], want[5])):
        assert torch.equal(a, b)
