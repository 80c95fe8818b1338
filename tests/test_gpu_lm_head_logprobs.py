"""fgm_lm_head_logprobs on a GPU against a plain 64-bit form.

Most cases take hidden rows and embeddings of small integers over 64: every
product and partial sum is a multiple of 2^-12 below 2^11 and exact in fp32, so
the logits are exact, many of them tie, and the tolerances are those of the
logits' own test (dz = 0). Normal inputs: D = 2816 products add up in fp32, each
addition off by at most 2^-23 of a partial sum below S = max sum |h e|:
dz = 2816 * 2^-23 S; the top words are compared where they are planted further
apart than that.
"""

import numpy as np
import pytest
import torch

import plain64
from test_gpu_logprobs import compare

pytestmark = pytest.mark.gpu
H = 2816


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def ws(fgm):
    return fgm.Workspace("cuda", nbytes=max(fgm.lm_head_logprobs_workspace_bytes(n, 262144, 16) for n in (8, 300, 2100)))


def integers(shape, seed, top):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randint(-top, top + 1, shape, generator=g, device="cuda").float() / 64).bfloat16()


def logits64(emb, h):
    """fp64 logits of the given rows (torch products in 64 bits)."""
    return torch.cat([h.double() @ emb[i:i + 32768].double().t() for i in range(0, emb.shape[0], 32768)], dim=1).cpu().numpy()


def run(fgm, ws, emb, h, tokens, k, T, **kw):
    r = fgm.lm_head_logprobs(emb, h, torch.tensor(tokens, dtype=torch.int32, device="cuda"), k=k, T=T, ws=ws, **kw)
    torch.cuda.synchronize()
    assert ws.status() == 0
    return r


@pytest.mark.parametrize("N,V,k,T", [
    (1, 1, 1, 1.0), (1, 5, 3, 1.0), (3, 255, 4, 0.5), (5, 256, 8, 1.0), (8, 257, 16, 1.0), (2, 1000, 0, 1.0), (100, 513, 2, 1.0),
    (127, 4099, 5, 1.0), (128, 4099, 1, 2.0), (129, 3000, 3, 1.0), (255, 2000, 7, 1.0), (256, 1025, 16, 1.0), (257, 700, 2, 0.7),
    (300, 20011, 4, 1.0), (513, 9000, 1, 1.0), (2050, 300, 3, 1.0), (5, 50021, 16, 1.0), (1, 40000, 9, 1.0)])
def test_exact_logits(fgm, ws, N, V, k, T):
    """Ragged rows and words, ties everywhere: ids equal, values to the sums' rounding."""
    emb, h = integers((V, H), V, 3), integers((N, H), N + 1, 4)
    g = torch.Generator().manual_seed(N)
    tokens = torch.randint(0, V, (N,), generator=g).tolist()
    if N > 2:
        tokens[1], tokens[2] = V, -1          # outside the vocabulary
    r = run(fgm, ws, emb, h, tokens, k, T)
    compare(r, logits64(emb, h), tokens, k, T)


@pytest.mark.parametrize("N,k", [(1, 8), (5, 8), (8, 3), (300, 4)])
def test_full_vocabulary(fgm, ws, N, k):
    V = 262144
    g = torch.Generator(device="cuda").manual_seed(N)
    emb = (torch.randn(V, H, generator=g, device="cuda") * 0.02).bfloat16()
    pick = torch.randint(0, V, (N, 10), generator=g, device="cuda")
    h = torch.randn(N, H, generator=g, device="cuda") * 0.2
    for i in range(10):
        h += (12.0 - i) / 1.126 * emb[pick[:, i]].float()
    h = h.bfloat16()
    tokens = pick[:, 2].tolist()
    r = run(fgm, ws, emb, h, tokens, k, 1.0)
    z = logits64(emb, h)
    S = float((h.double().abs() @ emb[:4096].double().abs().t()).max()) * 1.5
    top = np.sort(z, axis=1)[:, ::-1][:, :k + 1]
    dz = H * 2.0 ** -23 * S
    if (top[:, :-1] - top[:, 1:]).min() > 2 * dz:
        compare(r, z, tokens, k, 1.0, dz=dz)
    else:      # words closer than the sums' rounding may change places
        ids = r.top_ids.cpu().numpy()
        assert (np.take_along_axis(z, ids, 1) >= top[:, k - 1:k] - 2 * dz).all()
        compare(fgm.LogProbs(r.logp, r.entropy, None, None), z, tokens, 0, 1.0, dz=dz)
    # The first values of the logits carry the tensor pipe's truncation: 176
    # additions of 16 products, each off by at most an ulp of its sum, below
    # 2^-23 of S (sums of mixed signs stay below S). The row's largest are
    # computed again in fp32 (88 products a lane and a tree of 6: 2^-24 S each
    # and in truth far less); what the rest adds to ln l is weighted by their
    # share of the sum, at most 1: a bound of 176 * 2^-23 times their own size,
    # below the 13th largest logit.
    lp = plain64.logprobs(z, tokens, 0, 1.0)[0]
    rest = float(np.abs(np.sort(z, axis=1)[:, :-12]).max())
    err = np.abs(r.logp.cpu().double().numpy() - lp).max()
    print(f"N={N}: logp off by at most {err:.2e}")
    assert err <= 94 * 2.0 ** -24 * S + 176 * 2.0 ** -23 * rest + 2.0 ** -18


def test_rows_stand_alone_and_repeat(fgm, ws):
    """A row's results do not depend on its neighbours beyond the split of the
    words, and the same call gives the same bits."""
    V = 30000
    emb, h = integers((V, H), 1, 3), integers((700, H), 2, 4)
    tokens = list(range(700))
    a, b = run(fgm, ws, emb, h, tokens, 4, 1.0), run(fgm, ws, emb, h, tokens, 4, 1.0)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    one = run(fgm, ws, emb, h[600:601].contiguous(), [600], 4, 1.0)
    assert torch.equal(one.top_ids, a.top_ids[600:601]) and abs(float(one.logp[0] - a.logp[600])) < 2.0 ** -18


def test_agrees_with_argmax_and_logits(fgm, ws):
    """Beside lm_head_argmax on the same rows, in a graph replayed with other rows."""
    import synth
    emb = synth.embedding(32, vocab=50021, device="cuda")
    h = synth.hidden_states(41, 6, device="cuda")
    am = fgm.lm_head_argmax(emb, h, ws=ws)
    r = fgm.lm_head_logprobs(emb, h, am, k=2, ws=ws)
    assert torch.equal(r.top_ids[:, 0], am) and torch.equal(r.top_logp[:, 0], r.logp)
    assert r.logp.dtype == torch.float32 and (r.entropy > 0).all()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        am2 = fgm.lm_head_argmax(emb, h, ws=ws)
        r2 = fgm.lm_head_logprobs(emb, h, am2, k=3, ws=ws)
    for seed in (42, 43):
        h.copy_(synth.hidden_states(seed, 6, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r2.top_ids[:, 0], am2) and torch.equal(r2.top_logp[:, 0], r2.logp)
        z = logits64(emb, h)
        lp = plain64.logprobs(z, am2.tolist(), 0, 1.0)[0]
        S = float((h.double().abs() @ emb[:4096].double().abs().t()).max()) * 1.5
        assert np.abs(r2.logp.cpu().double().numpy() - lp).max() < 94 * 2.0 ** -24 * S + 176 * 2.0 ** -23 * np.abs(z).max() + 2.0 ** -18
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r3 = fgm.lm_head_logprobs(emb, h, am2, k=3, stream=s)
    s.synchronize()
    assert torch.equal(r3.logp, r2.logp) and torch.equal(r3.top_ids, r2.top_ids)


def test_nan_hidden_row_stays_apart(fgm, ws):
    emb, h = integers((3000, H), 1, 3), integers((9, H), 2, 4)
    ref = run(fgm, ws, emb, h, [5] * 9, 2, 1.0)
    h[4, 100] = float("nan")
    r = fgm.lm_head_logprobs(emb, h, torch.full((9,), 5, dtype=torch.int32, device="cuda"), k=2, ws=ws)
    torch.cuda.synchronize()
    assert ws.status() == fgm.STATUS_NONFINITE_LOGITS
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    assert torch.isnan(r.logp[4]) and torch.isnan(r.entropy[4])
    for x, y in zip(r, ref):
        assert torch.equal(x[keep], y[keep])


def test_refusals(fgm, ws):
    emb, h = integers((300, H), 1, 3), integers((4, H), 2, 4)
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    E = fgm.FgmError
    for be, bh in ((emb.float(), h), (emb[:, :100], h), (emb.cpu(), h), (emb, h.float()), (emb, h[:, :100]), (emb, h[0]),
                   (emb, h.cpu()), (emb.t(), h), (emb, torch.zeros(8, H, dtype=torch.bfloat16, device="cuda")[::2])):
        with pytest.raises(E):
            fgm.lm_head_logprobs(be, bh, t, ws=ws)
    for kw in (dict(k=-1), dict(k=17), dict(T=0.0), dict(T=float("nan")), dict(tokens=t[:2]), dict(tokens=t.long())):
        a = dict(tokens=t)
        a.update(kw)
        with pytest.raises(E):
            fgm.lm_head_logprobs(emb, h, ws=ws, **a)
    with pytest.raises(E):
        fgm.lm_head_logprobs(emb[:3], h, t, k=4, ws=ws)
    with pytest.raises(E):
        fgm.lm_head_logprobs(emb, h, t, ws=fgm.Workspace("cuda"))
    assert ws.status() == 0
