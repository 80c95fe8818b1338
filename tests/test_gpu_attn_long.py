"""fgm_attn_fwd where one CTA sees many tokens of a row, against plain 64-bit
forms computed on the device.

Tolerances, per element, with P the row's probabilities, A = sum P |v|, V = 448
times the largest scale of a block of values, n the row's tokens and U = n / 128
rounded up (the kernel's units):
  * a probability is held to 2^-8 of itself or, times its block's scale, 2^-34 of
    the largest: 2^-8 A + n 2^-34 max P V;
  * f16 on the way and the exponentials: 2^-12 A and 2^-20 A; the row sum adds U
    terms a thread and 12 more in fp32: (U + 12) 2^-24 A; an output adds 32 tokens
    at a time, 4 times a unit, in fp32 with truncation: 4 U 2^-23 A;
  * scores: ds = 2^-21 qmax sum|k| + D 2^-23 sum|q k|, times the scale, on P: 2 ds A;
  * the output is rounded to bf16: 2^-8 of itself.
lse: |err| <= ds + 2^-20 + (U + 12) 2^-24 + 2^-22 |lse|.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu
BLOCK = 64


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


def codes(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def make_cache(fgm, k, v, ks, vs):
    """k, v [blocks, H, 64, D] fp32 in units of the scales [blocks, H]."""
    n, H, _, D = k.shape
    return fgm.KVCache(codes(k).view(n, H, BLOCK, D // 64, 64).transpose(2, 3).contiguous(),
                       codes(v).transpose(2, 3).contiguous(), ks, vs)


def values(c, blocks, h):
    """K and V [tokens, D] of a head's blocks, fp64."""
    k = c.k_q[blocks, h].view(torch.float8_e4m3fn).double() * c.k_s[blocks, h].double()[:, None, None, None]
    v = c.v_q[blocks, h].view(torch.float8_e4m3fn).double() * c.v_s[blocks, h].double()[:, None, None]
    D = v.shape[1]
    return k.transpose(1, 2).reshape(-1, D), v.transpose(1, 2).reshape(-1, D)


def check_rows(out, lse, q, k, v, V, scale):
    """Rows out, q [R, D] and lse [R] that see all of k, v [n, D]; returns the largest |err| / |out|."""
    n, D = k.shape
    q, got, gl = q.double(), out.double(), lse.double()
    s = q @ k.t() * scale
    want_l = torch.logsumexp(s, dim=1)
    P = torch.exp(s - want_l[:, None])
    want = P @ v
    A = P @ v.abs()
    units = (n + 127) // 128
    ds = (2.0 ** -21 * q.abs().amax(dim=1) * k.abs().sum(dim=1).max()
          + D * 2.0 ** -23 * (q.abs() @ k.abs().t()).amax(dim=1)) * scale
    rel = 2.0 ** -8 + 2.0 ** -12 + 2.0 ** -20 + (units + 12) * 2.0 ** -24 + 4 * units * 2.0 ** -23 + 2 * ds[:, None]
    tol = rel * A + n * 2.0 ** -34 * P.amax(dim=1, keepdim=True) * V + 2.0 ** -8 * want.abs()
    err = (got - want).abs()
    worst = float((err / want.abs()).max())
    assert (err <= tol).all(), (worst, float((err / tol).max()))
    el = (gl - want_l).abs()
    assert (el <= ds + 2.0 ** -20 + (units + 12) * 2.0 ** -24 + 2.0 ** -22 * want_l.abs()).all(), float(el.max())
    return worst


@pytest.mark.parametrize("n,sink,D,G,M", [
    (8192, "zero", 64, 1, 1), (32768, "zero", 64, 1, 1), (32749, "zero", 128, 4, 5), (9001, "zero", 256, 8, 8),
    (32768, "like", 64, 1, 1), (262144, "like", 64, 1, 1)])
def test_attention_sink(fgm, n, sink, D, G, M):
    """A first token 15 nats above a body of small spread, its value zero or like
    the others'. 160 sequences read the same blocks, so that a CTA has a sequence
    to itself."""
    B = 160
    g = torch.Generator(device="cuda").manual_seed(n + D)
    nb = (n + BLOCK - 1) // BLOCK
    k = torch.randn(nb, 1, BLOCK, D, generator=g, device="cuda") * (0.3 * 64 * 8 / D ** 0.5)
    k[0, 0, 0] = 15.0 / 8 * 64 * 64 / D
    v = 200 + 60 * torch.randn(nb, 1, BLOCK, D, generator=g, device="cuda").clamp(-3, 3)
    if sink == "zero":
        v[0, 0, 0] = 0.0
    c = make_cache(fgm, k, v, torch.full((nb, 1), 2.0 ** -6, device="cuda"), torch.full((nb, 1), 2.0 ** -8, device="cuda"))
    q = (1 + 0.05 * torch.randn(B, M, G, D, generator=g, device="cuda")).bfloat16()
    tab = torch.arange(nb, dtype=torch.int32, device="cuda").repeat(B, 1)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    lse = torch.empty(B, M, G, device="cuda")
    ws = fgm.Workspace("cuda", nbytes=fgm.attn_workspace_bytes(B, M, G, 1, D))
    out = fgm.attn_fwd(c, q, lens, 0.125, block_table=tab, lse=lse, ws=ws)
    assert ws.status() == 0
    kv = values(c, slice(0, nb), 0)
    worst = 0.0
    for i in range(M):                              # row i sees the tokens up to its own
        seen = n - M + i + 1
        for b in range(0, B, 16):
            worst = max(worst, check_rows(out[b:b + 16, i].reshape(-1, D), lse[b:b + 16, i].reshape(-1),
                                          q[b:b + 16, i].reshape(-1, D), kv[0][:seen], kv[1][:seen], 448 * 2.0 ** -8, 0.125))
    print(f"n={n} {sink} D={D} rows={M * G}: output off by at most {worst:.2e} of itself")


def test_widest_products_of_a_full_batch(fgm):
    """1,024 sequences of 64 rows a kv head at D = 256: the most shared memory that
    operands and lengths take, which leaves the keys a single stage."""
    B, M, G, D = 1024, 8, 8, 256
    g = torch.Generator(device="cuda").manual_seed(8)
    nb = 16
    scale = torch.full((nb, 1), 2.0 ** -6, device="cuda")
    c = make_cache(fgm, torch.randn(nb, 1, BLOCK, D, generator=g, device="cuda") * 16,
                   torch.randn(nb, 1, BLOCK, D, generator=g, device="cuda") * 60, scale, scale)
    q = torch.randn(B, M, G, D, generator=g, device="cuda").bfloat16()
    tab = torch.stack([torch.randperm(nb, generator=g, device="cuda")[:6] for _ in range(B)]).to(torch.int32)
    lens = torch.randint(M, 6 * BLOCK + 1, (B,), generator=g, device="cuda").to(torch.int32)
    ws = fgm.Workspace("cuda", nbytes=fgm.attn_workspace_bytes(B, M, G, 1, D))
    lse = torch.empty(B, M, G, device="cuda")
    out = fgm.attn_fwd(c, q, lens, 0.0625, block_table=tab, lse=lse, ws=ws)
    assert ws.status() == 0
    for b in range(0, B, 31):
        k, v = values(c, tab[b].long(), 0)
        for i in range(M):
            seen = int(lens[b]) - M + i + 1
            check_rows(out[b, i], lse[b, i], q[b, i], k[:seen], v[:seen], 448 * 2.0 ** -6, 0.0625)


def test_many_units_a_cta(fgm):
    """Eight sequences of about 65,000 tokens with four heads: 108 units of 128
    tokens a CTA, more than three rounds of 32 block scales. Scales differ from
    block to block, keys are small enough that every token counts."""
    B, H, D, G, M = 8, 4, 64, 2, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = [65536 - 61 * b for b in range(B)]
    per = 1024
    n = B * per
    ks = torch.pow(2.0, torch.randint(-9, -5, (n, H), generator=g, device="cuda").float())
    vs = torch.pow(2.0, torch.randint(-9, -5, (n, H), generator=g, device="cuda").float())
    k = torch.randn(n, H, BLOCK, D, generator=g, device="cuda") * 24
    v = 60 + 20 * torch.randn(n, H, BLOCK, D, generator=g, device="cuda").clamp(-2, 2)
    c = make_cache(fgm, k, v, ks, vs)
    del k, v
    tab = torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(B, per)
    q = torch.randn(B, M, H * G, D, generator=g, device="cuda").bfloat16()
    ws = fgm.Workspace("cuda", nbytes=fgm.attn_workspace_bytes(B, M, H * G, H, D))
    lse = torch.empty(B, M, H * G, device="cuda")
    out = fgm.attn_fwd(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.25, block_table=tab, lse=lse, ws=ws)
    assert ws.status() == 0
    for b in range(B):
        for h in range(H):
            kk, vv = values(c, tab[b].long(), h)
            for i in range(M):
                seen = lens[b] - M + i + 1
                at = slice(h * G, (h + 1) * G)
                check_rows(out[b, i, at], lse[b, i, at], q[b, i, at], kk[:seen], vv[:seen], 448 * 2.0 ** -6, 0.25)


@pytest.mark.parametrize("n", [1, 64, 200])
@pytest.mark.parametrize("scale", [1e28, 1e32, 1e36])
def test_scores_far_below_zero(fgm, n, scale):
    """Every score equal and hugely negative: the mean of the values, whatever the size of the scores."""
    D, k0 = 64, -1.0
    nb = (n + BLOCK - 1) // BLOCK
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.full((nb, 1, BLOCK, D), k0, device="cuda")
    v = torch.randint(1, 16, (nb, 1, BLOCK, D), generator=g, device="cuda").float()
    one = torch.ones(nb, 1, device="cuda")
    c = make_cache(fgm, k, v, one, one)
    q = torch.full((1, 1, 1, D), 0.5, device="cuda").bfloat16()
    lse = torch.empty(1, 1, 1, device="cuda")
    ws = fgm.Workspace("cuda", nbytes=fgm.attn_workspace_bytes(1, 1, 1, 1, D))
    out = fgm.attn_fwd(c, q, torch.tensor([n], dtype=torch.int32, device="cuda"), scale, lse=lse, ws=ws)
    vals = values(c, slice(0, nb), 0)[1][:n]
    want = vals.mean(dim=0)
    # (equal scores: no error in P but the probabilities' 2^-8 and the sums')
    assert ((out[0, 0, 0].double() - want).abs() <= (2.0 ** -7 + 2.0 ** -12) * want).all()
    s = -0.5 * D * float(torch.tensor(scale, dtype=torch.float32))
    assert abs(float(lse) - s) <= 2.0 ** -21 * abs(s)
    assert ws.status() == 0


def test_windows_beyond_32_bits(fgm):
    """A window of any size is taken as it is."""
    g = torch.Generator(device="cuda").manual_seed(1)
    one = torch.full((4, 1), 2.0 ** -6, device="cuda")
    c = make_cache(fgm, torch.randn(4, 1, BLOCK, 64, generator=g, device="cuda") * 20,
                   torch.randn(4, 1, BLOCK, 64, generator=g, device="cuda") * 20, one, one)
    q = torch.randn(1, 2, 2, 64, generator=g, device="cuda").bfloat16()
    lens = torch.tensor([250], dtype=torch.int32, device="cuda")
    ref = fgm.attn_fwd(c, q, lens, 0.125)
    for window in (2 ** 31, 2 ** 32 + 5, 2 ** 40):
        assert torch.equal(fgm.attn_fwd(c, q, lens, 0.125, window=window), ref)
    for window in (-1, -2 ** 32, 3 - 2 ** 32):
        with pytest.raises(fgm.FgmError):
            fgm.attn_fwd(c, q, lens, 0.125, window=window)


@pytest.mark.parametrize("n", [200, 5000])
def test_block_scales_of_values_far_apart(fgm, n):
    """Blocks of zeros (scale 2^-60) between loud ones, 2^80 apart: the zeros keep
    their weight, in one CTA and over several."""
    H, G, M, D, B = 1, 2, 3, 64, 3
    g = torch.Generator(device="cuda").manual_seed(n)
    nb = (n + BLOCK - 1) // BLOCK
    quiet = torch.arange(nb, device="cuda") % 2 == 0
    k = torch.randn(nb, H, BLOCK, D, generator=g, device="cuda") * 24
    v = torch.where(quiet[:, None, None, None], torch.zeros((), device="cuda"),
                    200 + 60 * torch.randn(nb, H, BLOCK, D, generator=g, device="cuda").clamp(-3, 3))
    ks = torch.full((nb, H), 2.0 ** -6, device="cuda")
    vs = torch.where(quiet, 2.0 ** -60, 2.0 ** 20)[:, None].float().contiguous()
    c = make_cache(fgm, k, v, ks, vs)
    q = torch.randn(B, M, H * G, D, generator=g, device="cuda").bfloat16()
    tab = torch.arange(nb, dtype=torch.int32, device="cuda").repeat(B, 1)
    lse = torch.empty(B, M, H * G, device="cuda")
    ws = fgm.Workspace("cuda", nbytes=fgm.attn_workspace_bytes(B, M, H * G, H, D))
    out = fgm.attn_fwd(c, q, torch.full((B,), n, dtype=torch.int32, device="cuda"), 0.125, block_table=tab, lse=lse, ws=ws)
    assert ws.status() == 0
    kk, vv = values(c, slice(0, nb), 0)
    for b in range(B):
        for i in range(M):
            seen = n - M + i + 1
            check_rows(out[b, i], lse[b, i], q[b, i], kk[:seen], vv[:seen], 448 * 2.0 ** 20, 0.125)
