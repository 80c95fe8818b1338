"""fgm_logprobs on a GPU against a plain 64-bit form.

Tolerances, with X = max |z| / T over the row's logits within 200 T of its
largest (the others add less than 2^-288):
  * top ids: equal (the logits are compared as they are);
  * logp and top_logp: a term exp((z - m) / T) carries the rounding of m c and of
    the fused product, 2^-23 X of its exponent, and 2^-22 of the exponential; a
    sum of n terms over 256 lanes at 32 a chunk adds at most 2^-24 for each of
    16 + n / 8192 + 24 additions in line, below 2^-18 at n <= 262,144; the
    result adds (z - m) / T, at most 2 X, and ln l, each rounded once:
    |err| <= 2^-18 + 2^-22 + 2^-20 X + 2^-22 (|logp| + ln V);
  * entropy: the same relative errors on l and on sum e d, whose quotient is at
    most 2 X: |err| <= (2^-18 + 2^-20 X) (1 + entropy + ln V).
"""

import numpy as np
import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def ws(fgm):
    return fgm.Workspace("cuda", nbytes=fgm.logprobs_workspace_bytes(64, 262144, 16))


def check(fgm, ws, z, tokens, k, T, status=0, **kw):
    r = fgm.logprobs(z, torch.tensor(tokens, dtype=torch.int32, device="cuda"), k=k, T=T, ws=ws, **kw)
    torch.cuda.synchronize()
    assert ws.status() == status
    compare(r, z.cpu().double().numpy(), tokens, k, T)
    return r


def compare(r, z, tokens, k, T, dz=0.0):
    """dz: how far the logits themselves may be off."""
    V = z.shape[1]
    lp, ent, ids, tlp = plain64.logprobs(z, tokens, k, T)
    zz = np.where(np.isnan(z), -np.inf, z)
    with np.errstate(invalid="ignore"):
        X = (np.where(np.isfinite(zz) & (zz >= zz.max(axis=1, keepdims=True) - 200 * T), np.abs(zz), 0).max(axis=1) + dz) / T
    # what exceeds fp32 rounds to an infinity there
    lp, tlp = (np.where(x < -3.4028235677973366e38, -np.inf, x) for x in (lp, tlp))
    base = 2.0 ** -18 + 2.0 ** -22 + 2.0 ** -20 * X + 4 * dz / T

    def near(got, want, tol, what):
        got = got.cpu().double().numpy()
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=what)
        np.testing.assert_array_equal(np.isneginf(got), np.isneginf(want), err_msg=what)
        fin = np.isfinite(want)
        err = np.abs(np.where(fin, got, 0) - np.where(fin, want, 0))
        assert (err <= tol).all(), (what, err.max(), np.argmax(err - tol))

    near(r.logp, lp, base + 2.0 ** -22 * (np.where(np.isfinite(lp), np.abs(lp), 0) + np.log(V)), "logp")
    e = np.where(np.isnan(ent), 0, ent)
    near(r.entropy, ent, (2.0 ** -18 + 2.0 ** -20 * X + 4 * dz / T) * (1 + e + np.log(V)), "entropy")
    if k:
        np.testing.assert_array_equal(r.top_ids.cpu().numpy(), ids)
        near(r.top_logp, tlp, (base[:, None] + 2.0 ** -22 * (np.where(np.isfinite(tlp), np.abs(tlp), 0) + np.log(V))), "top_logp")
    else:
        assert r.top_ids is None and r.top_logp is None


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,k,T", [
    (1, 1, 1, 1.0), (3, 2, 2, 0.5), (5, 7, 3, 1.0), (2, 16, 16, 2.0), (9, 33, 5, 1.0), (4, 255, 0, 1.0), (7, 1000, 8, 0.7),
    (3, 4099, 16, 1.0), (2, 8191, 1, 1.0), (2, 16384, 8, 1.0), (5, 50021, 4, 1.3), (5, 262144, 8, 1.0), (1, 262143, 16, 0.3)])
def test_matches_plain(fgm, ws, dt, N, V, k, T):
    g = torch.Generator(device="cuda").manual_seed(V + N)
    z = torch.randn(N, V, generator=g, device="cuda") * 3
    z[:, torch.randint(0, V, (max(1, V // 50),), generator=g, device="cuda")] = float("-inf") if V > 40 else 0.5
    tokens = torch.randint(0, V, (N,), generator=g, device="cuda").tolist()
    check(fgm, ws, z.to(DT[dt]), tokens, k, T)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,k", [(701, 1, 1), (1300, 2, 2), (700, 5, 3), (900, 31, 16), (1217, 129, 0), (5000, 300, 4), (700, 715, 16),
                                   (4867, 1021, 3), (2000, 4099, 8)])
def test_many_short_rows(fgm, dt, N, V, k):
    """More rows than CTAs run at a time, short enough for a warp each; among them
    rows that tie throughout, that hold infinities and NaN, or nothing else."""
    g = torch.Generator().manual_seed(N + V)
    z = (torch.randn(N, V, generator=g) * 2).to(DT[dt])
    z[3] = 1.5                                 # ties everywhere
    z[5, 1:] = float("-inf")
    z[7] = float("-inf")
    z[11, V // 2] = float("nan")
    z[13, V - 1] = float("inf")
    z[17] = float("nan")
    z[19] = torch.finfo(DT[dt]).min
    if V > 80:
        z[23, ::2] = 9.0                       # more ties for the first places than a list of candidates holds
    tokens = torch.randint(-1, V + 1, (N,), generator=g).tolist()
    ws = fgm.Workspace("cuda", nbytes=fgm.logprobs_workspace_bytes(N, V, k))
    check(fgm, ws, z.cuda(), tokens, k, 0.9, status=fgm.STATUS_NONFINITE_LOGITS)


@pytest.mark.parametrize("T", [2.95e-39, 1e-38, 1e-30, 1e-6, 1e-3, 0.05, 1e4, 1e30])
@pytest.mark.parametrize("N,V", [(3, 1000), (2, 70001)])
def test_extreme_temperatures(fgm, ws, N, V, T):
    """From a one-hot to a uniform distribution. Differences from the largest
    logit carry 2^-24 of themselves and their product with log2(e) / T 2^-22, up
    to 200 binary places down: e |d| <= 0.54, so a term's error is below 2^-22 of
    the sum and the bounds need no part that grows with |z| / T, but the given
    token's own (z - m) / T: |err| <= 2^-18 + 2^-22 (|logp| + ln V)."""
    g = torch.Generator().manual_seed(V)
    z = torch.randn(N, V, generator=g) * 3 + 9
    top = z.argmax(dim=1)
    z[0, 5] = z[0, top[0]]                     # a tie for the first place
    tokens = [int(top[0]), 7, int(top[2])][:N] if N == 3 else [int(top[0]), int(top[1])]
    r = fgm.logprobs(z.cuda(), torch.tensor(tokens, dtype=torch.int32, device="cuda"), k=4, T=T, ws=ws)
    assert ws.status() == 0
    T32 = float(np.float32(T))
    lp, ent, ids, tlp = plain64.logprobs(z.double().numpy(), tokens, 4, T32)
    np.testing.assert_array_equal(r.top_ids.cpu().numpy(), ids)
    for got, want in ((r.logp, lp), (r.top_logp, tlp), (r.entropy, ent)):
        got = got.cpu().double().numpy()
        want = np.where(want < -3.4028235677973366e38, -np.inf, want)
        fin = np.isfinite(want)
        np.testing.assert_array_equal(got[~fin], want[~fin])
        assert (np.abs(got[fin] - want[fin]) <= 2.0 ** -18 + 2.0 ** -22 * (np.abs(want[fin]) + np.log(V))).all(), (got, want)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_rows_of_any_alignment_and_distance(fgm, ws, dt):
    """Views whose rows start at every offset within 16 bytes; what lies between the rows is not read as logits."""
    g = torch.Generator(device="cuda").manual_seed(5)
    buf = torch.full((6, 12345), float("nan"), device="cuda").to(DT[dt])
    for off in range(9):
        z = buf[:, off:off + 9001]
        z.copy_((torch.randn(6, 9001, generator=g, device="cuda") * 2).to(DT[dt]))
        check(fgm, ws, z, [0, 9000, 1, 8999, 4096, 7], 6, 1.0)
        buf.fill_(float("nan"))


def test_many_rows(fgm):
    """More rows than CTAs at a time, no split; row results do not depend on their neighbours."""
    g = torch.Generator(device="cuda").manual_seed(6)
    z = torch.randn(5000, 777, generator=g, device="cuda") * 2
    ws = fgm.Workspace("cuda", nbytes=fgm.logprobs_workspace_bytes(5000, 777, 3))
    tokens = torch.randint(0, 777, (5000,), generator=g, device="cuda").tolist()
    r = check(fgm, ws, z, tokens, 3, 1.0)
    one = check(fgm, ws, z[4321:4322], [tokens[4321]], 3, 1.0)
    assert torch.equal(one.logp, r.logp[4321:4322]) and torch.equal(one.entropy, r.entropy[4321:4322])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_ties_and_orders(fgm, ws, dt):
    """Equal logits go to the lower index; rising and falling rows; few distinct values."""
    V = 30011
    g = torch.Generator(device="cuda").manual_seed(8)
    rows = [torch.zeros(V), torch.full((V,), -7.5), torch.arange(V) / V * 8, -torch.arange(V) / V * 8,
            torch.randint(0, 3, (V,), generator=torch.Generator().manual_seed(1)).float(),
            torch.where(torch.arange(V) % 3 == 0, 0.0, -0.0),
            torch.full((V,), float("-inf")).index_fill(0, torch.tensor([5, 20000]), 1.0)]
    z = torch.stack(rows).cuda().to(DT[dt])
    check(fgm, ws, z, [0, V - 1, 3, 4, 5, 6, 20000], 16, 1.0)
    del g


def test_lowest_values_infinities_and_nan(fgm, ws):
    V = 9000
    g = torch.Generator(device="cuda").manual_seed(9)
    base = torch.randn(1, V, generator=g, device="cuda")
    low = torch.finfo(torch.float32).min
    z = base.repeat(3, 1)
    z[0, 100:8900] = low                                   # masked with the type's lowest value
    z[1, 1:] = low                                         # a single word left
    z[2] = low                                             # nothing but masked words: uniform
    r = check(fgm, ws, z, [0, 5, 77], 4, 1.0)
    assert abs(float(r.logp[2]) + np.log(V)) < 1e-5 and abs(float(r.entropy[2]) - np.log(V)) < 1e-5
    zb = torch.full((2, V), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16, device="cuda")
    zb[0, 7] = 2.0
    check(fgm, ws, zb, [7, 8], 3, 0.5)
    z = base.repeat(4, 1) * 30
    z[0, 17] = float("nan")                                # counts as -inf
    z[1] = float("-inf")                                   # no distribution
    z[2, 44] = float("inf")
    z[3] = float("nan")
    check(fgm, ws, z, [17, 3, 44, 5], 5, 1.0, status=fgm.STATUS_NONFINITE_LOGITS)
    z = torch.full((1, 40), 3.0e38, device="cuda")
    z[0, 3] = 3.3e38
    check(fgm, ws, z, [3], 2, 1.0)


def test_tokens_outside_and_optional_outputs(fgm, ws):
    g = torch.Generator(device="cuda").manual_seed(10)
    z = torch.randn(4, 12000, generator=g, device="cuda")
    check(fgm, ws, z, [-1, 12000, 2 ** 31 - 1, 11999], 2, 1.0)
    t = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda")
    full = fgm.logprobs(z, t, k=3, ws=ws)
    r = fgm.logprobs(z, k=3, ws=ws)
    assert r.logp is None and torch.equal(r.entropy, full.entropy) and torch.equal(r.top_logp, full.top_logp)
    r = fgm.logprobs(z, t, entropy=False, ws=ws)
    assert r.entropy is None and r.top_ids is None and torch.equal(r.logp, full.logp)
    out = fgm.LogProbs(torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(4, 3, dtype=torch.int32, device="cuda"),
                       torch.zeros(4, 3, device="cuda"))
    r = fgm.logprobs(z, t, k=3, out=out, ws=ws)
    assert r is out and torch.equal(out.top_ids, full.top_ids) and torch.equal(out.logp, full.logp)


def test_logits_of_a_verify_step(fgm, ws):
    """The logits that lm_head_sample returns, scored at its temperature: the
    argmax is the first alternative, and on a graph's replay with new logits too."""
    import synth
    emb = synth.embedding(32, vocab=50021, device="cuda")
    h = synth.hidden_states(77, 5, device="cuda")
    am = torch.empty(5, dtype=torch.int32, device="cuda")
    u = torch.full((5,), 0.5, device="cuda")
    _, z = fgm.lm_head_sample(emb, h, 0.8, am[:4].clone().fill_(3), u[:4], u, argmax=am, ws=ws)
    r = fgm.logprobs(z, am, k=4, T=0.8, ws=ws)
    assert torch.equal(r.top_ids[:, 0], am) and torch.equal(r.top_logp[:, 0], r.logp)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rg = fgm.logprobs(z, am, k=4, T=0.8, ws=ws)
    for seed in (1, 2):
        z.copy_(torch.randn(z.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        compare(rg, z.cpu().double().numpy(), am.tolist(), 4, 0.8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r2 = fgm.logprobs(z, am, k=4, T=0.8, stream=s)        # its own workspace, on another stream
    s.synchronize()
    assert torch.equal(r2.logp, rg.logp) and torch.equal(r2.top_ids, rg.top_ids)


def test_logits_offsets_beyond_32_bits(fgm, ws):
    """Rows that start past 2^32 elements."""
    z = torch.empty(3, 2 ** 31 + 5, dtype=torch.bfloat16, device="cuda")[:, :5000]
    z.copy_(torch.randn(3, 5000, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda"))
    check(fgm, ws, z, [1, 2, 3], 4, 1.0)


def test_refusals(fgm, ws):
    z = torch.zeros(2, 100, device="cuda")
    t = torch.zeros(2, dtype=torch.int32, device="cuda")
    E = fgm.FgmError
    for bad in (z.double(), z[0], z.cpu(), z.t(), z[:1].expand(2, 100), z.int()):
        with pytest.raises(E):
            fgm.logprobs(bad, t, ws=ws)
    for bt in (t.long(), t[:1], t.cpu(), torch.zeros(2, 1, dtype=torch.int32, device="cuda")):
        with pytest.raises(E):
            fgm.logprobs(z, bt, ws=ws)
    for k in (-1, 17, 101):
        with pytest.raises(E):
            fgm.logprobs(z, t, k=k, ws=ws)
    with pytest.raises(E):
        fgm.logprobs(z[:, :3], t, k=4, ws=ws)
    for T in (0.0, -1.0, float("inf"), float("nan"), 1e-39):
        with pytest.raises(E):
            fgm.logprobs(z, t, T=T, ws=ws)
    small = fgm.Workspace("cuda")
    with pytest.raises(E):
        fgm.logprobs(torch.zeros(1, 262144, device="cuda"), t[:1], k=4, ws=small)
    with pytest.raises(E):
        fgm.logprobs(z, t, k=2, out=fgm.LogProbs(t.float(), t.float(), None, None), ws=ws)
    with pytest.raises(E):
        fgm.logprobs(z, t, out=fgm.LogProbs(t.double(), t.float(), None, None), ws=ws)
    with pytest.raises(E):
        fgm.logprobs(torch.zeros(0, 5, device="cuda"), ws=ws)
    assert ws.status() == 0
