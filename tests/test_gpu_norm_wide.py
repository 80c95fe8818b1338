"""Block norms of 13 to 16 warps a row, on either side of where the kernel for the usual types ends."""

import pytest
import torch

from test_gpu_block_norm import B, F, check, fgm, gate_of, rows  # noqa: F401 (fgm: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [3064, 3080, 3592, 4088, 4096, 4104])
@pytest.mark.parametrize("h_type", [F, B])
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
def test_types_and_gates(fgm, D, h_type, gate):
    g = torch.Generator(device="cuda").manual_seed(D)
    N = 1111
    post, pre = (torch.rand(D, generator=g, device="cuda") + 0.5 for _ in range(2))
    h, y = rows(N, D, h_type, g, 2.0), rows(N, D, B, g)
    kw = dict(gate=gate_of(gate, N, D, B, g), a=0.7, b=-1.3, offset=1.0)
    check(fgm, h, y, post=post, pre=pre, **kw)
    check(fgm, h, y, post=post, pre_norm=False, **kw)
    check(fgm, h, y, pre=pre, post_norm=False, **kw)


@pytest.mark.parametrize("D", [3080, 4096])
def test_in_place_and_again(fgm, D):
    g = torch.Generator(device="cuda").manual_seed(9)
    h, y = rows(900, D, B, g), rows(900, D, B, g)
    o, n = check(fgm, h, y)
    for _ in range(3):
        h1, y1 = h.clone(), y.clone()
        fgm.block_norm(h1, y1, h_out=h1, xn=y1)
        assert torch.equal(h1, o) and torch.equal(y1, n)
