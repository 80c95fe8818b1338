"""Head counts whose rows a kv head pass 32 bits: refused like any other above
FGM_ATTN_MAX_ROWS. Nothing here reaches a GPU."""

import ctypes

import pytest

import fine_grained_moe_gb300 as fgm
from test_kv_abi import AT, attn, cache, lib    # noqa: F401


@pytest.mark.parametrize("n_q_heads", [1 << 29, 1 << 28, (1 << 30) + 8, 2 ** 31 - 1])
@pytest.mark.parametrize("M", [1, 2, 4, 8])
def test_rows_beyond_32_bits(lib, n_q_heads, M):    # noqa: F811
    assert fgm.attn_workspace_bytes(1, M, n_q_heads, 1, 64) == 0
    assert attn(lib, cache(n_kv_heads=1), Hq=n_q_heads, M=M, stride=n_q_heads * 64) == -1
    assert b"above" in lib.fgm_last_error()


@pytest.mark.parametrize("M", range(1, 9))
def test_rows_at_their_limit(lib, M):    # noqa: F811
    most = 64 // M
    assert fgm.attn_workspace_bytes(1, M, most * 3, 3, 128) > 0
    assert fgm.attn_workspace_bytes(1, M, (most + 1) * 3, 3, 128) == 0
