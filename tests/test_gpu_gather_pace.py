"""Gathered rows in tiles of very different sizes, one after the other: warps that have
rows in some of them only."""

import pytest
import torch

from test_gpu_grouped_gemm import check, fgm, ragged, weights  # noqa: F401 (fgm: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("N,K", [(600, 64), (300, 1040), (1500, 2816)])
def test_tiles_of_one_row_and_of_many(fgm, kind, N, K):
    g = torch.Generator(device="cuda").manual_seed(N)
    counts = [1, 300, 2, 8, 129, 1, 1, 40, 0, 256, 16, 17, 1, 255, 3, 33] * 6
    off = ragged(counts)
    x = torch.randn(1000, K, generator=g, device="cuda").bfloat16()
    w, s = weights(len(counts), N, K, kind, g)
    rows = torch.randint(0, 1000, (off[-1],), generator=g, device="cuda", dtype=torch.int32)
    ws = fgm.Workspace("cuda", nbytes=fgm.grouped_gemm_workspace_bytes(1000, off[-1], len(counts), N, K))
    at = torch.tensor(off, dtype=torch.int32, device="cuda")
    out = fgm.grouped_gemm(x, w, s, at, rows=rows, ws=ws)
    assert ws.status() == 0
    check(out, x, w, s, off, rows=rows.long())
    for _ in range(20):
        assert torch.equal(fgm.grouped_gemm(x, w, s, at, rows=rows, ws=ws), out)
    assert ws.status() == 0
