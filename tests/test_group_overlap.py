"""Grouping's outputs lie apart from the ids that it reads and from each other. Nothing here
reaches a GPU."""

import os

import pytest
import torch

import fine_grained_moe_gb300 as fgm

AT = 1 << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fgm.LIB_PATH):
        from fine_grained_moe_gb300 import build
        build.build()
    return fgm.lib()


def group(lib, ids, off, order, n=1000, E=128):
    return lib.fgm_moe_group(ids, n, E, off, order, AT, 1 << 50, None)


@pytest.mark.parametrize("ids,off,order", [
    (0, 1 << 20, 0), (0, 1 << 20, 3996), (0, 1 << 20, -3996), (0, 0, 1 << 20), (0, 3996, 1 << 20), (516, 4, 1 << 20), (0, 1 << 20, (1 << 20) + 512),
    (0, (1 << 20) + 3996, 1 << 20)])
def test_overlaps(lib, ids, off, order):
    assert group(lib, AT + ids, AT + off, AT + order) == -1 and b"overlap" in lib.fgm_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="host addresses must not reach a GPU")
@pytest.mark.parametrize("ids,off,order", [(0, 4000, 4516), (4000, 8000, 0), (516, 0, 4516)])
def test_neighbours(lib, ids, off, order):
    assert group(lib, AT + ids, AT + off, AT + order) in (-3, -4)
