"""Products grouped by expert against 64 bits: ragged groups, gathered rows, both weight types."""

import math

import pytest
import torch

import prompt64 as p64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


def weights(E, N, K, kind, g):
    w = torch.randn(E, N, K, generator=g, device="cuda") * 0.05
    if kind == "bf16":
        return w.bfloat16(), None
    s = w.abs().amax(dim=2) / 448
    return (w / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def check(out, x, w, s, offsets, src=None, rows=None):
    """Every row of some expert; x already gathered where src is None."""
    E, N = w.shape[:2]
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            xe = x[a:b] if rows is None else x[rows[a:b]]
            val = p64.e4m3(w[e]) if w.dtype == torch.uint8 else w[e].double()
            sc = torch.ones(N, dtype=torch.float64, device="cuda") if s is None else s[e].double()
            want, err = p64.products(xe, val, sc, w.dtype == torch.uint8)
            p64.within(out[a:b], want, p64.rounded(want, err, torch.bfloat16))


def ragged(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return off


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("N,K", [(1, 16), (8, 32), (31, 48), (96, 128), (129, 144), (256, 1408), (300, 272), (704, 2816), (2816, 704), (520, 4400)])
@pytest.mark.parametrize("counts", [(1,), (0, 3, 0, 17, 0), (33, 1, 0, 64, 65), (300, 0, 5, 130)])
def test_products(fgm, kind, N, K, counts):
    g = torch.Generator(device="cuda").manual_seed(N + K)
    off = ragged(counts)
    R = off[-1]
    x = torch.randn(R, K, generator=g, device="cuda")
    x[:, ::53] *= 20
    x = x.bfloat16()
    w, s = weights(len(counts), N, K, kind, g)
    ws = fgm.Workspace("cuda", nbytes=fgm.grouped_gemm_workspace_bytes(R, R, len(counts), N, K))
    out = fgm.grouped_gemm(x, w, s, torch.tensor(off, dtype=torch.int32, device="cuda"), ws=ws)
    assert ws.status() == 0
    check(out, x, w, s, off)


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("T,per,E,N,K", [(1, 8, 128, 64, 64), (5, 8, 128, 704, 2816), (77, 2, 16, 200, 160), (401, 1, 3, 136, 96), (600, 4, 1, 2112, 1408)])
def test_gathered_rows(fgm, kind, T, per, E, N, K):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = (torch.randn(T, K, generator=g, device="cuda") * torch.exp(torch.randn(T, 1, generator=g, device="cuda") * 3)).bfloat16()
    w, s = weights(E, N, K, kind, g)
    ids = torch.randint(0, E, (T * per,), generator=g, device="cuda", dtype=torch.int32)
    off, order = fgm.moe_group(ids, E)
    out = fgm.grouped_gemm(x, w, s, off, rows=order, per=per)
    check(out, x, w, s, off.tolist(), rows=(order // per).long())


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_rows_of_no_expert_stay(fgm, kind):
    g = torch.Generator(device="cuda").manual_seed(2)
    E, N, K, T = 6, 72, 64, 100
    w, s = weights(E, N, K, kind, g)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    off = torch.tensor([3, 10, 10, 40, 41, 41, 83], dtype=torch.int32, device="cuda")
    out = torch.full((T, N), 9.0, dtype=torch.bfloat16, device="cuda")
    fgm.grouped_gemm(x, w, s, off, out=out)
    assert (out[:3] == 9).all() and (out[83:] == 9).all()
    check(out, x, w, s, off.tolist())
    # no rows at all, and offsets beyond the rows, which are taken within them
    out.fill_(9.0)
    fgm.grouped_gemm(x, w, s, torch.full((E + 1,), 50, dtype=torch.int32, device="cuda"), out=out)
    assert (out == 9).all()
    fgm.grouped_gemm(x, w, s, torch.tensor([-5, 20, 20, 20, 20, 20, 1000], dtype=torch.int32, device="cuda"), out=out)
    check(out, x, w, s, [0, 20, 20, 20, 20, 20, T])
    fgm.grouped_gemm(x, w, s, torch.tensor([90, 20, 7, 7, 7, 7, 7], dtype=torch.int32, device="cuda"), out=out.fill_(9.0))
    assert (out == 9).all()


def test_rows_outside_x_are_zero(fgm):
    g = torch.Generator(device="cuda").manual_seed(3)
    for kind in ("e4m3", "bf16"):
        w, s = weights(2, 40, 64, kind, g)
        x = torch.randn(10, 64, generator=g, device="cuda").bfloat16()
        x[0] = math.nan                            # (what such a row takes in its place is not seen)
        rows = torch.tensor([4, -1, 20, 9, 2**31 - 1, -2**31, 19, 3], dtype=torch.int32, device="cuda")
        off = torch.tensor([0, 5, 8], dtype=torch.int32, device="cuda")
        out = fgm.grouped_gemm(x, w, s, off, rows=rows, per=2)
        gone = torch.tensor([1, 2, 4, 5], device="cuda")
        assert (out[gone] == 0).all()
        keep = [i for i in range(8) if i not in gone.tolist()]
        full = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
        full[keep] = x[(rows[keep] // 2).long()]
        check(out, full, w, s, off.tolist())


def test_non_finite_rows_and_weights(fgm):
    g = torch.Generator(device="cuda").manual_seed(4)
    w, s = weights(1, 33, 96, "e4m3", g)
    x = torch.randn(9, 96, generator=g, device="cuda").bfloat16()
    x[2, 5], x[4, 90], x[6] = math.nan, math.inf, 0
    w[0, 7, 11] = 0x7F
    off = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    out = fgm.grouped_gemm(x, w, s, off)
    assert out[[2, 4]].isnan().all() and out[:, 7].isnan().all()
    rest = [i for i in range(33) if i != 7]
    assert out[[0, 1, 3, 5, 7, 8]][:, rest].isfinite().all() and (out[6][rest] == 0).all()


def test_small_and_large_values(fgm):
    g = torch.Generator(device="cuda").manual_seed(5)
    w, s = weights(2, 64, 128, "e4m3", g)
    x = torch.randn(40, 128, generator=g, device="cuda") * torch.logspace(-30, 30, 40, device="cuda")[:, None]
    x = x.bfloat16()
    x[:, 3] *= 64                                  # an element far above its row's others
    off = torch.tensor([0, 19, 40], dtype=torch.int32, device="cuda")
    check(fgm.grouped_gemm(x, w, s, off), x, w, s, off.tolist())


def test_rows_apart_and_odd_outputs(fgm):
    g = torch.Generator(device="cuda").manual_seed(6)
    w, s = weights(3, 64, 160, "e4m3", g)
    wide = torch.randn(70, 200, generator=g, device="cuda").bfloat16()
    x = wide[:, 24:184]
    off = torch.tensor([0, 30, 31, 70], dtype=torch.int32, device="cuda")
    check(fgm.grouped_gemm(x, w, s, off), x, w, s, off.tolist())
    # an output that is not 16-byte aligned
    room = torch.zeros(70 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    out = room[1:].view(70, 64)
    fgm.grouped_gemm(x, w, s, off, out=out)
    check(out, x, w, s, off.tolist())
    assert room[0] == 0


@pytest.mark.parametrize("K", [8, 24, 56, 72, 200, 1000])
def test_bf16_rows_that_end_inside_a_step(fgm, K):
    """16 elements of K are a step of the products; what lies behind K, here infinities, is not read."""
    g = torch.Generator(device="cuda").manual_seed(K)
    w, _ = weights(3, 50, K, "bf16", g)
    wide = torch.full((90, K + 64), math.inf, dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = torch.randn(90, K, generator=g, device="cuda").bfloat16()
    x = wide[:, :K]
    off = torch.tensor([0, 30, 33, 90], dtype=torch.int32, device="cuda")
    check(fgm.grouped_gemm(x, w, None, off), x, w, None, off.tolist())
    rows = torch.randperm(90, generator=g, device="cuda").int()
    check(fgm.grouped_gemm(x, w, None, off, rows=rows), x, w, None, off.tolist(), rows=rows.long())


@pytest.mark.parametrize("K", [16, 48, 112, 1040])
def test_e4m3_rows_that_end_inside_a_step(fgm, K):
    g = torch.Generator(device="cuda").manual_seed(K)
    w, s = weights(3, 50, K, "e4m3", g)
    wide = torch.full((90, K + 64), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = torch.randn(90, K, generator=g, device="cuda").bfloat16()
    x = wide[:, :K]
    off = torch.tensor([0, 30, 33, 90], dtype=torch.int32, device="cuda")
    check(fgm.grouped_gemm(x, w, s, off), x, w, s, off.tolist())


def test_the_same_bits_again(fgm):
    g = torch.Generator(device="cuda").manual_seed(7)
    w, s = weights(20, 320, 512, "e4m3", g)
    x = torch.randn(900, 512, generator=g, device="cuda").bfloat16()
    off, order = fgm.moe_group(torch.randint(0, 20, (900,), generator=g, device="cuda", dtype=torch.int32), 20)
    a = fgm.grouped_gemm(x, w, s, off, rows=order)
    for _ in range(3):
        assert torch.equal(a, fgm.grouped_gemm(x, w, s, off, rows=order))


def test_many_experts_and_long_rows(fgm):
    g = torch.Generator(device="cuda").manual_seed(8)
    w, s = weights(1024, 24, 32, "e4m3", g)
    counts = torch.randint(0, 4, (1024,), generator=torch.Generator().manual_seed(1)).tolist()
    off = ragged(counts)
    x = torch.randn(off[-1], 32, generator=g, device="cuda").bfloat16()
    check(fgm.grouped_gemm(x, w, s, torch.tensor(off, dtype=torch.int32, device="cuda")), x, w, s, off)


def test_outputs_behind_32_bits(fgm):
    """2^31 elements of output and more: the last rows are where they belong."""
    g = torch.Generator(device="cuda").manual_seed(9)
    N, K, R = 2816, 16, 770_000
    w, s = weights(1, N, K, "e4m3", g)
    x = torch.randn(R, K, generator=g, device="cuda").bfloat16()
    out = fgm.grouped_gemm(x, w, s, torch.tensor([0, R], dtype=torch.int32, device="cuda"))
    for a in (0, R // 2, R - 300):
        check(out[a:a + 300], x[a:a + 300], w, s, [0, 300])


def test_binding_refusals(fgm):
    g = torch.Generator(device="cuda").manual_seed(1)
    w, s = weights(2, 16, 32, "e4m3", g)
    x = torch.randn(4, 32, device="cuda").bfloat16()
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for call in (lambda: fgm.grouped_gemm(x.float(), w, s, off), lambda: fgm.grouped_gemm(x[:, :16], w, s, off), lambda: fgm.grouped_gemm(x, w.int(), s, off),
                 lambda: fgm.grouped_gemm(x, w, s[:1], off), lambda: fgm.grouped_gemm(x, w, s, off[:2]), lambda: fgm.grouped_gemm(x, w, s, off, per=0),
                 lambda: fgm.grouped_gemm(x, w, s, off, rows=off.long()), lambda: fgm.grouped_gemm(x, w, s, off, out=torch.empty(4, 8, device="cuda")),
                 lambda: fgm.grouped_gemm(x, w[..., :24].contiguous(), s, off), lambda: fgm.grouped_gemm(x[:0], w, s, off),
                 lambda: fgm.grouped_gemm(x, w.cpu(), s, off)):
        with pytest.raises(fgm.FgmError):
            call()
