"""The cache, its attention, the MoE layers and the log probabilities together,
as a decoding loop uses them: a prompt written into the caches of two layers,
then verify steps of five tokens whose drafts are partly taken back, each step
one captured graph. Every operator is compared with its plain 64-bit form on
the inputs that it had in the run, with the tolerances of its own test file
(the lm_head's: 2816 products added in fp32, each addition within 2^-23 of a
partial sum below S = max sum |h e|).
"""

import numpy as np
import pytest
import torch

import oracle
import plain64
import synth
from helpers import REL_TOL, rowwise_rel_err, to_oracle_layer
from test_gpu_kv_cache import check_attn, host, random_cache, shuffled_table
from test_gpu_lm_head_logprobs import logits64
from test_gpu_logprobs import compare

pytestmark = pytest.mark.gpu
HIDDEN, HEADS, GROUP, D, M = 2816, 2, 4, 128, 5
SCALE = D ** -0.5


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


class Mixer:
    """A layer's projections (the caller's part) and its cache."""

    def __init__(self, fgm, seed):
        g = torch.Generator().manual_seed(seed)
        wide = (HEADS * GROUP + 2 * HEADS) * D
        self.w_in = (torch.randn(HIDDEN, wide, generator=g) / HIDDEN ** 0.5).bfloat16().cuda()
        self.w_out = (torch.randn(HEADS * GROUP * D, HIDDEN, generator=g) / (HEADS * GROUP * D) ** 0.5).bfloat16().cuda()
        self.cache = random_cache(fgm, 9, HEADS, D, seed)
        self.table = shuffled_table(1, 8, 9, seed).cuda()

    def split(self, x):
        """q, k, v of x's tokens: slices of one product's rows."""
        n = x.shape[0]
        z = (x @ self.w_in).unsqueeze(0)
        a, b = HEADS * GROUP * D, (HEADS * GROUP + HEADS) * D
        return (z[..., :a].view(1, n, HEADS * GROUP, D), z[..., a:b].view(1, n, HEADS, D),
                z[..., b:].view(1, n, HEADS, D))


def test_prompt_and_verify_steps(fgm):
    V = 20011
    mixers = [Mixer(fgm, 5), Mixer(fgm, 6)]
    layers = [synth.layer(i, device="cuda", s=1.1) for i in range(2)]
    emb = synth.embedding(33, vocab=V, device="cuda")
    ws = fgm.Workspace("cuda", nbytes=max(fgm.attn_workspace_bytes(1, M, HEADS * GROUP, HEADS, D),
                                          fgm.lm_head_logprobs_workspace_bytes(M, V, 3), fgm.workspace_bytes(M, V)))
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")

    def tokens(n, seed):
        return torch.cat([synth.hidden_states(seed + i, min(8, n - i), device="cuda") for i in range(0, n, 8)])

    # the prompt, a layer at a time (its hidden states stand in for the layers' own)
    length = 203
    lens.fill_(length)
    for i, mx in enumerate(mixers):
        _, k, v = mx.split(tokens(length, 900 + i * 300))
        kq, vq, ks, vs = host(mx.cache)
        fgm.kv_append(mx.cache, k, v, lens, block_table=mx.table, ws=ws)
        plain64.append_side(kq, ks, k.cpu().double().numpy(), [length], mx.table.tolist())
        plain64.append_side(vq, vs, v.cpu().double().numpy(), [length], mx.table.tolist())
        torch.cuda.synchronize()
        for got, want in zip(host(mx.cache), (kq, vq, ks, vs)):
            if got.dtype == np.uint8:
                got, want = np.where(got == 0x80, 0, got), np.where(want == 0x80, 0, want)
            np.testing.assert_array_equal(got, want)

    x = torch.zeros(M, HIDDEN, dtype=torch.bfloat16, device="cuda")
    draft = torch.zeros(M, dtype=torch.int32, device="cuda")

    def step():
        h, kept = x, []
        for mx, layer in zip(mixers, layers):
            q, k, v = mx.split(h)
            fgm.kv_append(mx.cache, k, v, lens, block_table=mx.table, ws=ws)
            lse = torch.empty(1, M, HEADS * GROUP, device="cuda")
            o = fgm.attn_fwd(mx.cache, q, lens, SCALE, block_table=mx.table, lse=lse, ws=ws)
            mixed = h + o.view(M, -1) @ mx.w_out
            y = fgm.moe_layer_fwd(layer, mixed, ws=ws)
            h = mixed + y
            kept.append((q, k, v, o, lse, mixed, y))
        best = fgm.lm_head_argmax(emb, h, ws=ws)
        return kept, h, best, fgm.lm_head_logprobs(emb, h, draft, k=3, T=0.8, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    before = [host(m.cache) for m in mixers]
    with torch.cuda.stream(side):                    # (libraries choose their kernels outside the capture)
        lens.fill_(length + M)
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for mx, (kq, vq, ks, vs) in zip(mixers, before):
        mx.cache.k_q.copy_(torch.from_numpy(plain64.k_cached(kq)))
        mx.cache.v_q.copy_(torch.from_numpy(np.ascontiguousarray(vq.transpose(0, 1, 3, 2))))
        mx.cache.k_s.copy_(torch.from_numpy(ks))
        mx.cache.v_s.copy_(torch.from_numpy(vs))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept, h, best, lp = step()

    for n, accepted in enumerate((3, 5, 1, 2)):
        x.copy_(tokens(M, 40 + n))
        draft.copy_(torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(n)))
        lens.fill_(length + M)
        before = [host(m.cache) for m in mixers]
        graph.replay()
        torch.cuda.synchronize()
        assert ws.status() == 0
        for mx, layer, (kq, vq, ks, vs), (q, k, v, o, lse, mixed, y) in zip(mixers, layers, before, kept):
            tab = mx.table.tolist()
            plain64.append_side(kq, ks, k.cpu().double().numpy(), [length + M], tab)
            plain64.append_side(vq, vs, v.cpu().double().numpy(), [length + M], tab)
            for got, want in zip(host(mx.cache), (kq, vq, ks, vs)):
                if got.dtype == np.uint8:
                    got, want = np.where(got == 0x80, 0, got), np.where(want == 0x80, 0, want)
                np.testing.assert_array_equal(got, want)
            check_attn(o, lse, q, kq, vq, ks, vs, [length + M], tab, SCALE, 0)
            assert torch.isfinite(y).all()
        if n == 0:
            layer, mixed, y = layers[1], kept[1][5], kept[1][6]
            ref = oracle.moe_layer(to_oracle_layer(layer), mixed.cpu().double().numpy())
            assert (rowwise_rel_err(y, ref.y) <= REL_TOL).all()
        S = float((h.double().abs() @ emb.double().abs().t()).max())
        z = logits64(emb, h)
        compare(lp._replace(top_ids=None, top_logp=None), z, draft.tolist(), 0, 0.8, dz=HIDDEN * 2.0 ** -23 * S)
        assert torch.equal(lp.top_ids[:, 0], best)
        length += accepted
