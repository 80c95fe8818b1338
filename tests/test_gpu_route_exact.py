"""Routing against exact logits where K is not split (9,729 tokens and more)."""

import pytest

from test_gpu_route import check, fgm, inputs  # noqa: F401 (fgm: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [9728, 9729, 12_345, 16_381])
@pytest.mark.parametrize("bias", [False, True])
def test_tokens(fgm, T, bias):
    """9,728 tokens have their K cut in two, 9,729 have it whole."""
    x, w, b = inputs(T, T)
    check(fgm, x, w, b if bias else None)


@pytest.mark.parametrize("T", [9728, 9729])
@pytest.mark.parametrize("alike", [3, 40])
def test_many_near_experts(fgm, T, alike):
    x, w, b = inputs(T, 10 + alike)
    w[20:20 + alike] = w[20]
    b[20:20 + alike] = b[20] + (b.new_tensor(range(alike)) % 3) * 2.0 ** -20
    check(fgm, x, w, b)
    w[21:20 + alike:2, ::401] *= 1 + 2.0 ** -7
    check(fgm, x, w, b)


def test_equal_rows_take_the_lower_index(fgm):
    x, w, b = inputs(9729, 4)
    w[1::2] = w[::2]
    b[1::2] = b[::2]
    check(fgm, x, w, b)


def test_one_workspace_for_longer_and_shorter_prompts(fgm):
    """The largest call's workspace serves the others, one after the other."""
    ws = fgm.Workspace("cuda", nbytes=fgm.moe_route_workspace_bytes(9729))
    for T in (9729, 9728, 1664, 3, 1665, 9729):
        x, w, b = inputs(T, T)
        check(fgm, x, w, b, ws=ws)
