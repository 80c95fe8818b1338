"""The 8-bit KV cache on a GPU: fgm_kv_append and fgm_attn_fwd against plain
64-bit forms.

Tolerances.
  * append: the scale is a power of two and a code one rounding of x / s, which
    is exact in fp32; codes and scales are compared bit for bit.
  * attention, per element, with A = sum P|v|, V = max |v| of the row's tokens:
      - scores: a query element is held to 2^-21 of its row's largest (two E4M3
        terms, the second times 16, of q scaled to a largest element above 224:
        half a subnormal step is 2^-10, 2^-10 / 16 / 224 < 2^-21); D products
        add up in fp32, each add within 2^-23 of a sum below sum|q k|:
        ds = 2^-21 qmax sum|k| + D 2^-23 sum|q k|, both times the scale;
      - probabilities are rounded to f16, 2^-12 of themselves, and enter the
        product as two E4M3 terms: 2^-4 of 2^-4 = 2^-8 of themselves, and where the second term is subnormal 2^-10 / 32 / 32 =
        2^-20 of the largest that their CTA saw; a CTA holds at most 512 tokens
        of a row in these cases and the CTAs' largest sum to at most 1:
        512 * 2^-20 V;
      - exponentials and the sums of up to T terms: exp2 within 2^-21, sums in
        fp32, 2^-14 covers both at T <= 2^9 terms a partial;
      - the output is rounded to bf16: 2^-8 of itself.
    |err| <= (2^-8 + 2^-12 + 2^-14 + 2 ds) A + 2^-11 V + 2^-8 |out|.
  * lse: |err| <= ds + 2^-14 (1 + |lse| 2^-4).
"""

import numpy as np
import pytest
import torch

import oracle
import plain64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def ws(fgm):
    return fgm.Workspace("cuda", nbytes=max(fgm.attn_workspace_bytes(1024, 8, 8, 1, 256),
                                            fgm.attn_workspace_bytes(16, 1, 64, 1, 256)))


def random_cache(fgm, n_blocks, H, D, seed, fill=None):
    """A cache of random finite codes and power-of-two scales (or one code everywhere)."""
    g = torch.Generator().manual_seed(seed)
    c = fgm.KVCache.empty(n_blocks, H, D)
    for t in (c.k_q, c.v_q):
        code = torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8)
        code = torch.where((code & 0x7F) >= 0x78, code & 0x87, code)     # no NaN, no code above 240
        t.copy_(code if fill is None else torch.full_like(code, fill))
    for t in (c.k_s, c.v_s):
        t.copy_(torch.pow(2.0, torch.randint(-9, -5, t.shape, generator=g).float()))
    return c


def host(c):
    """[blocks, H, 64, D] codes of K and V, and the scales, on the host."""
    return (plain64.k_natural(c.k_q.cpu().numpy()), np.ascontiguousarray(c.v_q.cpu().numpy().transpose(0, 1, 3, 2)),
            c.k_s.cpu().numpy().copy(), c.v_s.cpu().numpy().copy())


def shuffled_table(B, per, n_blocks, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(n_blocks, generator=g)[:B * per].view(B, per).to(torch.int32)


def check_append(fgm, ws, c, k, v, lens, table, stream=None):
    kq, vq, ks, vs = host(c)
    tab = table.tolist() if table is not None else \
        [[b * (c.v_q.shape[0] // len(lens)) + j for j in range(c.v_q.shape[0] // len(lens))] for b in range(len(lens))]
    fgm.kv_append(c, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                  block_table=None if table is None else table.cuda(), ws=ws, stream=stream)
    torch.cuda.synchronize()
    plain64.append_side(kq, ks, k.cpu().double().numpy(), lens, tab)
    plain64.append_side(vq, vs, v.cpu().double().numpy(), lens, tab)
    got = host(c)
    for a, b, what in zip(got, (kq, vq, ks, vs), ("k codes", "v codes", "k scales", "v scales")):
        if a.dtype == np.uint8:      # a signed zero may differ in sign only
            a, b = np.where(a == 0x80, 0, a), np.where(b == 0x80, 0, b)
        np.testing.assert_array_equal(a, b, err_msg=what)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,N,lens", [
    (1, 1, [1]), (2, 1, [64]), (2, 1, [65]), (8, 5, [62]), (3, 5, [66]), (2, 8, [3]),      # lens < N: early tokens skipped
    (1, 4, [0]), (2, 63, [63]), (2, 64, [64]), (2, 64, [100]), (1, 130, [131]), (2, 200, [200, 333, 201]),
    (2, 7, [1, 0, 7, 64, 65, 129]),
])
def test_append_matches_plain(fgm, ws, D, H, N, lens):
    per = 6
    g = torch.Generator().manual_seed(N * 1000 + D + sum(lens))
    B = len(lens)
    c = random_cache(fgm, B * per + 2, H, D, seed=N + D)
    size = torch.exp(torch.randn(B, N, 1, 1, generator=g))       # some blocks grow, some do not
    k = (torch.randn(B, N, H, D, generator=g) * size).bfloat16().cuda()
    v = (torch.randn(B, N, H, D, generator=g) * size * 0.3).bfloat16().cuda()
    check_append(fgm, ws, c, k, v, lens, shuffled_table(B, per, B * per + 2, seed=D))
    assert ws.status() == 0


@pytest.mark.parametrize("a", [448.0, 450.0, 224.0, 2.0 ** -60 * 448, 2.0 ** -75, 1e-38, 0.0, 3e38, 7.0 * 2.0 ** 90])
def test_append_scale_at_its_steps(fgm, ws, a):
    """amax on, just above and far from 448 times a power of two."""
    c = random_cache(fgm, 2, 1, 64, seed=5)
    k = torch.zeros(1, 2, 1, 64)
    k[0, 0, 0, 3], k[0, 1, 0, 60] = a, -a / 3
    v = torch.full((1, 2, 1, 64), a)
    check_append(fgm, ws, c, k.bfloat16().cuda(), v.bfloat16().cuda(), [2], None)
    check_append(fgm, ws, c, v.bfloat16().cuda(), k.bfloat16().cuda(), [4], None)      # with kept tokens
    assert ws.status() == 0


def test_append_strided_views_and_token_by_token(fgm, ws):
    """K and V as slices of a fused projection's rows; one token at a time gives
    the cache of a plain form that was driven the same way."""
    H, D, Hq = 2, 128, 4
    g = torch.Generator().manual_seed(9)
    c = random_cache(fgm, 3, H, D, seed=1)
    for n, ln in ((5, 5), (1, 6), (1, 7), (60, 67), (3, 68)):      # the last call takes drafts back: 67 -> 65 kept
        qkv = torch.randn(1, n, (Hq + 2 * H) * D, generator=g).bfloat16().cuda()
        k = qkv[..., Hq * D:(Hq + H) * D].view(1, n, H, D)
        v = qkv[..., (Hq + H) * D:].view(1, n, H, D)
        check_append(fgm, ws, c, k, v, [ln], torch.tensor([[2, 0, 1]], dtype=torch.int32))
    assert ws.status() == 0


def test_append_nonfinite_values(fgm, ws):
    c = random_cache(fgm, 2, 1, 64, seed=7)
    k = torch.randn(1, 3, 1, 64, generator=torch.Generator().manual_seed(1))
    k[0, 0, 0, 1], k[0, 1, 0, 2], k[0, 2, 0, 3] = float("nan"), float("inf"), float("-inf")
    kb = k.bfloat16().cuda()
    check_append(fgm, ws, c, kb, torch.full_like(kb, float("nan")), [3], None)
    assert ws.status() == fgm.STATUS_NONFINITE_KV
    assert ws.status() == 0


def test_append_bad_tables_write_nothing(fgm, ws):
    """Blocks outside the cache, and lengths that no table holds."""
    for lens, table in (([5], [[2, 0]]), ([5], [[-1, 0]]), ([-3], [[0, 1]])):
        c = random_cache(fgm, 2, 2, 64, seed=11)
        before = host(c)
        k = torch.ones(1, 5, 2, 64, dtype=torch.bfloat16, device="cuda")
        fgm.kv_append(c, k, k, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      block_table=torch.tensor(table, dtype=torch.int32, device="cuda"), ws=ws)
        assert ws.status() == fgm.STATUS_BAD_BLOCK
        for a, b in zip(before, host(c)):
            np.testing.assert_array_equal(a, b)
    # too long for the table: the tokens that it has room for are written
    c, k = random_cache(fgm, 2, 2, 64, seed=11), torch.ones(1, 5, 2, 64, dtype=torch.bfloat16, device="cuda")
    fgm.kv_append(c, k, k, torch.tensor([130], dtype=torch.int32, device="cuda"), ws=ws)
    assert ws.status() == fgm.STATUS_BAD_BLOCK
    kq = host(c)[0]
    assert (oracle.e4m3_decode(kq[1, :, 61:]) * host(c)[2][1][:, None, None] == 1.0).all()


def attn_case(fgm, ws, c, q, lens, table, scale, window=0, stream=None, hide=True):
    """One call compared with the plain form; with hide, every slot that no row
    may see holds NaN codes."""
    B, M, Hq, D = q.shape
    tab = table.tolist()
    kq, vq, ks, vs = host(c)
    if hide:
        seen = np.zeros(kq.shape[:1] + (64,), bool)
        for b in range(B):
            lo = max(0, lens[b] - M - window + 1) if window else 0
            for t in range(lo, lens[b]):
                seen[tab[b][t // 64], t % 64] = True
        for nat, t in ((kq, c.k_q), (vq, c.v_q)):
            nan = np.where(seen[:, None, :, None], nat, 0x7F if t is c.k_q else 0xFF).astype(np.uint8)
            t.copy_(torch.from_numpy(plain64.k_cached(nan) if t is c.k_q else
                                     np.ascontiguousarray(nan.transpose(0, 1, 3, 2))))
    out = torch.full((B, M, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, M, Hq), 7.0, device="cuda")
    r = fgm.attn_fwd(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, block_table=table.cuda(),
                     window=window, out=out, lse=lse, ws=ws, stream=stream)
    torch.cuda.synchronize()
    assert r is out
    check_attn(out, lse, q, kq, vq, ks, vs, lens, tab, scale, window)
    return out, lse


def check_attn(out, lse, q, kq, vq, ks, vs, lens, tab, scale, window):
    D = q.shape[3]
    kv = oracle.e4m3_decode(kq) * ks.astype(np.float64)[:, :, None, None]
    vv = oracle.e4m3_decode(vq) * vs.astype(np.float64)[:, :, None, None]
    o, l, A, V, sqk, sk = plain64.attn(q.cpu().double().numpy(), kv, vv, lens, tab, scale, window)
    ds = 2.0 ** -21 * sk + D * 2.0 ** -23 * sqk
    go, gl = out.cpu().double().numpy(), lse.cpu().double().numpy()
    tol = (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -14 + 2 * ds[..., None]) * A + 2.0 ** -11 * V + 2.0 ** -8 * np.abs(o)
    assert np.isfinite(go).all()
    bad = np.abs(go - o) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], go[bad][:4], o[bad][:4], tol[bad][:4])
    empty = np.isneginf(l)
    np.testing.assert_array_equal(np.isneginf(gl), empty)
    assert (go[empty] == 0).all()
    err = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, l))
    lt = ds + 2.0 ** -14 * (1 + np.abs(np.where(empty, 0, l)) / 16)
    assert (err <= lt).all(), (err.max(), lt.min())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,G,M,lens,window", [
    (1, 1, 1, [1], 0), (2, 2, 1, [64], 0), (2, 2, 5, [65], 0), (1, 8, 5, [700], 0), (2, 8, 8, [131], 0),
    (8, 2, 3, [1000], 0), (1, 16, 4, [513], 0), (2, 3, 7, [129, 5, 0, 64, 63, 300], 0), (1, 64, 1, [100], 0),
    (2, 2, 5, [900], 64), (2, 2, 5, [900], 1), (1, 4, 8, [200, 3, 64, 130], 3), (2, 6, 4, [641], 65), (1, 2, 2, [300], 10 ** 9),
    (4, 1, 8, [4, 8, 9, 0], 0),
])
def test_attn_matches_plain(fgm, ws, D, H, G, M, lens, window):
    g = torch.Generator().manual_seed(D + M * 7 + sum(lens))
    per = max(1, (max(lens) + 63) // 64)
    n = len(lens) * per + 1
    c = random_cache(fgm, n, H, D, seed=D + M)
    q = (torch.randn(len(lens), M, H * G, D, generator=g) * 2).bfloat16().cuda()
    attn_case(fgm, ws, c, q, lens, shuffled_table(len(lens), per, n, seed=3), D ** -0.5, window)
    assert ws.status() == 0


def test_attn_many_short_and_one_long(fgm, ws):
    """Many sequences end inside a CTA's share; one spans many CTAs."""
    lens = [int(x) for x in np.random.RandomState(3).randint(0, 150, 90)] + [20000] + [0, 1]
    H, G, M, D = 2, 2, 2, 64
    tab = torch.zeros(len(lens), 313, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = (n + 63) // 64
        tab[b, :m] = torch.arange(at, at + m)
        at += m
    c = random_cache(fgm, at, H, D, seed=21)
    q = (torch.randn(len(lens), M, H * G, D, generator=torch.Generator().manual_seed(2)) * 2).bfloat16().cuda()
    a = attn_case(fgm, ws, c, q, lens, tab, 0.125, hide=False)
    b = attn_case(fgm, ws, c, q, lens, tab, 0.125, hide=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])        # no order of atomics in it
    assert ws.status() == 0


@pytest.mark.parametrize("H,G,M,D,B", [(1, 8, 8, 256, 260), (2, 8, 8, 128, 150), (1, 6, 8, 256, 200), (3, 4, 8, 64, 130),
                                       (1, 1, 1, 64, 1024)])
def test_attn_many_sequences_of_many_rows(fgm, H, G, M, D, B):
    """More (sequence, head)s than CTAs at the widest products, where a CTA goes
    through several with one or two query buffers; empty ones in between."""
    rs = np.random.RandomState(B)
    lens = [int(n) if e else 0 for n, e in zip(rs.randint(1, 300, B), rs.randint(0, 5, B))]
    tab = torch.zeros(B, 5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = (n + 63) // 64
        tab[b, :m] = torch.arange(at, at + m)
        at += m
    c = random_cache(fgm, at, H, D, seed=B)
    ws = fgm.Workspace("cuda", nbytes=fgm.attn_workspace_bytes(B, M, H * G, H, D))
    q = (torch.randn(B, M, H * G, D, generator=torch.Generator().manual_seed(B)) * 2).bfloat16().cuda()
    for window in (0, 70):
        attn_case(fgm, ws, c, q, lens, tab, D ** -0.5, window)
    assert ws.status() == 0


def test_attn_sink_and_extreme_scores(fgm, ws):
    """A first token far above a flat body; scores of hundreds; uneven block scales."""
    H, G, M, D, L = 1, 4, 5, 128, 3000
    g = torch.Generator().manual_seed(4)
    c = random_cache(fgm, 48, H, D, seed=8)
    kq = plain64.k_natural(c.k_q.cpu().numpy())
    kq[0, 0, 0] = 0x70                                                 # 128 in every dim
    c.k_q.copy_(torch.from_numpy(plain64.k_cached(kq)))
    c.k_s.mul_(0.25)
    c.v_s.copy_(torch.pow(2.0, torch.randint(-40, 20, c.v_s.shape, generator=g).float()))
    q = (torch.randn(1, M, G, D, generator=g) * 0.5 + 0.3).bfloat16().cuda()
    tab = torch.arange(48, dtype=torch.int32).view(1, 48)
    for scale in (0.088, 5.0, 1e-3):
        attn_case(fgm, ws, c, q, [L], tab, scale)
    assert ws.status() == 0


def test_attn_shared_prefix_and_strided_queries(fgm, ws):
    """Two sequences read the same physical blocks; q is a slice of a fused projection."""
    H, G, M, D = 2, 2, 3, 64
    c = random_cache(fgm, 6, H, D, seed=2)
    tab = torch.tensor([[4, 1, 0], [4, 1, 3]], dtype=torch.int32)
    qkv = torch.randn(2, M, (H * G + 2 * H) * D, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    q = qkv[..., :H * G * D].view(2, M, H * G, D)
    attn_case(fgm, ws, c, q, [150, 140], tab, 0.125, hide=False)


def test_attn_nonfinite_query_rows_stay_apart(fgm, ws):
    c = random_cache(fgm, 3, 1, 64, seed=2)
    q = torch.randn(1, 3, 2, 64, generator=torch.Generator().manual_seed(3)).bfloat16()
    ref = fgm.attn_fwd(c, q.cuda(), torch.tensor([130], dtype=torch.int32, device="cuda"), 0.125, ws=ws)
    q[0, 1, 0, 5], q[0, 2, 1, 6] = float("nan"), float("inf")
    out = fgm.attn_fwd(c, q.cuda(), torch.tensor([130], dtype=torch.int32, device="cuda"), 0.125, ws=ws)
    nan = torch.zeros(1, 3, 2, dtype=torch.bool)
    nan[0, 1, 0] = nan[0, 2, 1] = True
    assert torch.equal(torch.isnan(out.cpu()).all(-1), nan) and torch.equal(torch.isnan(out.cpu()).any(-1), nan)
    assert torch.equal(out.cpu()[~nan], ref.cpu()[~nan])


def test_attn_bad_tables_are_reported(fgm, ws):
    c = random_cache(fgm, 3, 1, 64, seed=2)
    q = torch.randn(1, 2, 2, 64).bfloat16().cuda()
    for lens, table in (([100], [[0, 9]]), ([100], [[-5, 1]]), ([200], [[0, 1]]), ([-1], [[0, 1]])):
        fgm.attn_fwd(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.125,
                     block_table=torch.tensor(table, dtype=torch.int32, device="cuda"), ws=ws)
        assert ws.status() == fgm.STATUS_BAD_BLOCK, (lens, table)


def test_cache_offsets_beyond_32_bits(fgm, ws):
    """Blocks whose codes start past 2^32 bytes."""
    H, D = 8, 256
    n = 2 ** 32 // (H * D * 64) + 40
    c = fgm.KVCache.empty(n, H, D)
    last = torch.tensor([[n - 1, n - 7, n - 30]], dtype=torch.int32)
    small = random_cache(fgm, 3, H, D, seed=4)
    for name in ("k_q", "v_q", "k_s", "v_s"):
        getattr(c, name)[last[0].long()] = getattr(small, name)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(1, 4, H, D, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(1, 4, 2 * H, D, generator=g).bfloat16().cuda()
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    here = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    fgm.kv_append(c, k, v, lens, block_table=last.cuda(), ws=ws)
    fgm.kv_append(small, k, v, lens, block_table=here, ws=ws)
    for name in ("k_q", "v_q", "k_s", "v_s"):
        assert torch.equal(getattr(c, name)[last[0].long()], getattr(small, name)), name
    a = fgm.attn_fwd(c, q, lens, 0.0625, block_table=last.cuda(), ws=ws)
    b = fgm.attn_fwd(small, q, lens, 0.0625, block_table=here, ws=ws)
    assert torch.equal(a, b)


def test_streams_graphs_and_own_workspace(fgm):
    """On a side stream without a workspace, and captured: replays follow lengths
    and queries changed in place, two graphs alternate on one workspace."""
    H, G, M, D = 2, 4, 5, 128
    c = random_cache(fgm, 20, H, D, seed=2)
    g = torch.Generator().manual_seed(6)
    q = torch.randn(1, M, H * G, D, generator=g).bfloat16().cuda()
    k, v = (torch.randn(1, M, H, D, generator=g).bfloat16().cuda() for _ in range(2))
    tab = torch.arange(20, dtype=torch.int32).view(1, 20)
    tab_d, lens = tab.cuda(), torch.tensor([500], dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = fgm.attn_fwd(c, q, lens, 0.09, block_table=tab_d, stream=st)
    st.synchronize()
    ref = fgm.attn_fwd(c, q, lens, 0.09, block_table=tab_d)
    assert torch.equal(out, ref)
    ws = fgm.Workspace("cuda", nbytes=fgm.attn_workspace_bytes(1, M, H * G, H, D))
    outs, graphs = [torch.zeros_like(out) for _ in range(2)], []
    torch.cuda.synchronize()
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            fgm.kv_append(c, k, v, lens, block_table=tab_d, ws=ws)
            fgm.attn_fwd(c, q, lens, 0.09, block_table=tab_d, window=64 * i, out=outs[i], ws=ws)
        graphs.append(gr)
    for L in (505, 1277, 66, 5):
        lens.fill_(L)
        q.copy_(torch.randn(1, M, H * G, D, generator=g).bfloat16())
        for gr in graphs + graphs:
            gr.replay()
        torch.cuda.synchronize()
        kq, vq, ks, vs = host(c)
        for i in range(2):
            lse = torch.zeros(1, M, H * G, device="cuda")
            again = fgm.attn_fwd(c, q, lens, 0.09, block_table=tab_d, window=64 * i, lse=lse, ws=ws)
            assert torch.equal(again, outs[i])
            check_attn(outs[i], lse, q, kq, vq, ks, vs, [L], tab.tolist(), 0.09, 64 * i)
    assert ws.status() == 0


def test_append_then_attend_equals_attention_over_the_values(fgm, ws):
    """A prompt, then verify steps of which only some tokens are kept: the cache
    holds what a plain form of the same steps holds, and attention reads it."""
    H, G, D, gamma = 2, 2, 128, 4
    g = torch.Generator().manual_seed(12)
    c = random_cache(fgm, 8, H, D, seed=3)
    tab = shuffled_table(1, 7, 8, seed=5)
    length = 0
    for n, kept in ((190, 190), (5, 2), (5, 5), (5, 1), (5, 3), (5, 4), (5, 5)):
        k, v = (torch.randn(1, n, H, D, generator=g).bfloat16().cuda() for _ in range(2))
        check_append(fgm, ws, c, k, v, [length + n], tab)
        if n == gamma + 1:
            q = torch.randn(1, n, H * G, D, generator=g).bfloat16().cuda()
            attn_case(fgm, ws, c, q, [length + n], tab, D ** -0.5, hide=False)
        length += kept
    assert ws.status() == 0


def test_refusals(fgm, ws):
    c = random_cache(fgm, 4, 2, 64, seed=1)
    lens = torch.tensor([9], dtype=torch.int32, device="cuda")
    k = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    E = fgm.FgmError
    for bad in (k.float(), k[:, :, :1], k[..., :32], k.cpu(), k.transpose(2, 3), k[0]):
        with pytest.raises(E):
            fgm.kv_append(c, bad, bad, lens, ws=ws)
    with pytest.raises(E):
        fgm.kv_append(c, k, k[:, :2], lens, ws=ws)
    for bl in (lens.long(), torch.tensor([9, 9], dtype=torch.int32, device="cuda"), lens.cpu()):
        with pytest.raises(E):
            fgm.kv_append(c, k, k, bl, ws=ws)
        with pytest.raises(E):
            fgm.attn_fwd(c, q, bl, 0.1, ws=ws)
    for bt in (torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, device="cuda"),
               torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, 0, dtype=torch.int32, device="cuda")):
        with pytest.raises(E):
            fgm.attn_fwd(c, q, lens, 0.1, block_table=bt, ws=ws)
    for s in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(E):
            fgm.attn_fwd(c, q, lens, s, ws=ws)
    with pytest.raises(E):
        fgm.attn_fwd(c, q, lens, 0.1, window=-1, ws=ws)
    with pytest.raises(E):      # 9 tokens
        fgm.attn_fwd(c, torch.zeros(1, 9, 4, 64, dtype=torch.bfloat16, device="cuda"), lens, 0.1, ws=ws)
    with pytest.raises(E):      # 3 heads over 2 kv heads
        fgm.attn_fwd(c, torch.zeros(1, 1, 3, 64, dtype=torch.bfloat16, device="cuda"), lens, 0.1, ws=ws)
    with pytest.raises(E):      # 8 * 16 rows on a kv head
        fgm.attn_fwd(c, torch.zeros(1, 8, 32, 64, dtype=torch.bfloat16, device="cuda"), lens, 0.1, ws=ws)
    with pytest.raises(E):
        fgm.attn_fwd(c, q, lens, 0.1, out=torch.zeros_like(q[:, :2]), ws=ws)
    with pytest.raises(E):
        fgm.attn_fwd(c, q, lens, 0.1, lse=torch.zeros(1, 3, 4, dtype=torch.float64, device="cuda"), ws=ws)
    with pytest.raises(E):
        fgm.KVCache.empty(4, 2, 96)
    with pytest.raises(E):
        fgm.kv_append(fgm.KVCache(c.k_q, c.v_q, c.k_s, c.v_s.double()), k, k, lens, ws=ws)
    with pytest.raises(E):      # a token's heads 4 bytes off the 16-byte grid
        wide = torch.zeros(1, 3, 2 * 64 + 8, dtype=torch.bfloat16, device="cuda")
        off = wide[..., 2:2 + 128].view(1, 3, 2, 64)
        fgm.kv_append(c, off, off, lens, ws=ws)
    torch.cuda.synchronize()
    assert ws.status() == 0
