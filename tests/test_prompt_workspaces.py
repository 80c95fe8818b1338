"""Workspace sizes of the routing, grouping, grouped products and experts: what the
largest call is given serves every smaller one. Nothing here reaches a GPU."""

import ctypes
import os
import random

import pytest
import torch

import fine_grained_moe_gb300 as fgm

MOST = 1 << 18


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fgm.LIB_PATH):
        from fine_grained_moe_gb300 import build
        build.build()
    return fgm.lib()


def rises(sizes):
    return all(0 < a <= b for a, b in zip(sizes, sizes[1:]))


def test_routing_sizes_never_fall(lib):
    assert rises([lib.fgm_moe_route_workspace_bytes(T) for T in range(1, 21_000)])
    assert rises([lib.fgm_moe_route_workspace_bytes(T) for T in range(1, MOST + 1, 89)] + [lib.fgm_moe_route_workspace_bytes(MOST)])


@pytest.mark.parametrize("E", [1, 128, 1024])
def test_grouping_sizes_never_fall(lib, E):
    steps = [n + d for n in range(1024, 8 * MOST, 1024) for d in (-1, 0, 1)]
    assert rises([lib.fgm_moe_group_workspace_bytes(n, E) for n in sorted(set(steps)) if n <= 8 * MOST])
    assert rises([lib.fgm_moe_group_workspace_bytes(70_000, e) for e in range(1, 1025)])


def test_experts_sizes_never_fall(lib):
    around = [T + d for T in range(128, MOST, 128) for d in (-1, 0, 1)]
    assert rises([lib.fgm_moe_experts_workspace_bytes(T) for T in around])


def test_grouped_sizes_never_fall(lib):
    f = lib.fgm_grouped_gemm_workspace_bytes
    assert rises([f(n, n, 8, 64, 64) for n in range(1, 3000)]) and rises([f(77, 77, 8, 64, K) for K in range(8, 4096, 8)])
    assert f(77, 1, 1, 1, 64) == f(77, 1 << 20, 1024, 4096, 64)


@pytest.mark.skipif(torch.cuda.is_available(), reason="host addresses must not reach a GPU")
def test_a_workspace_for_the_largest_serves_the_smaller(lib):
    """What passes the checks is refused here for want of a GPU alone."""
    buf = (ctypes.c_uint8 * 8192)()
    at = (ctypes.addressof(buf) + 255) // 256 * 256
    rng = random.Random(3)
    pairs = [(9728, 9729), (4864, 9729), (1664, 1665), (1664, 16381), (32768, 32769), (5, MOST)]
    pairs += [tuple(sorted((int(2 ** rng.uniform(0, 18)), int(2 ** rng.uniform(0, 18))))) for _ in range(300)]
    for small, large in pairs:
        n = lib.fgm_moe_route_workspace_bytes(large)
        assert lib.fgm_moe_route(at, at, at, 2816, small, at, at, at, at, at, n, None) in (-3, -4), (small, large)
        n = lib.fgm_moe_group_workspace_bytes(8 * large, 128)
        assert lib.fgm_moe_group(at, 8 * small, 128, at + (1 << 40), at + (1 << 41), at, n, None) in (-3, -4), (small, large)


@pytest.mark.skipif(torch.cuda.is_available(), reason="host addresses must not reach a GPU")
def test_bf16_weights_need_no_room_for_terms(lib):
    at = 1 << 20
    call = lambda kind, n: lib.fgm_grouped_gemm(at, 64, 1 << 20, None, 1, at, at, kind, None, 3, 10, 64, at, 1 << 20, at, n, None)      # noqa: E731
    assert call(1, fgm.workspace_bytes(1)) in (-3, -4)
    assert call(1, fgm.workspace_bytes(1) - 256) == -2
    full = lib.fgm_grouped_gemm_workspace_bytes(1 << 20, 1 << 20, 3, 10, 64)
    assert call(3, fgm.workspace_bytes(1)) == -2 and call(3, full) in (-3, -4) and call(3, full - 256) == -2
