"""Host-side refusals of the KV-cache entry points: nothing here reaches a GPU."""

import ctypes
import os

import pytest
import torch

import fine_grained_moe_gb300 as fgm


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fgm.LIB_PATH):
        from fine_grained_moe_gb300 import build
        build.build()
    return fgm.lib()


BUF = (ctypes.c_uint8 * 8192)()
AT = (ctypes.addressof(BUF) + 255) // 256 * 256


def cache(**kw):
    f = dict(k_q=AT, k_s=AT, v_q=AT, v_s=AT, n_blocks=4, n_kv_heads=2, head_dim=64)
    f.update(kw)
    return fgm.fgm_kv_cache(**f)


def append(lib, c=None, k=AT, v=AT, stride=128, B=1, N=1, lens=AT, table=None, mb=4, ws=AT, nws=1 << 30):
    return lib.fgm_kv_append(None if c is False else ctypes.byref(c or cache()), k, v, stride, B, N, lens, table, mb, ws,
                             nws, None)


def attn(lib, c=None, q=AT, stride=256, B=1, M=1, Hq=4, lens=AT, table=None, mb=4, scale=0.1, window=0, out=AT, lse=None,
         ws=AT, nws=1 << 30):
    return lib.fgm_attn_fwd(None if c is False else ctypes.byref(c or cache()), q, stride, B, M, Hq, lens, table, mb,
                            scale, window, out, lse, ws, nws, None)


@pytest.mark.parametrize("bad", [
    dict(k_q=None), dict(v_q=AT + 8), dict(k_s=None), dict(v_s=AT + 2), dict(n_blocks=0), dict(n_blocks=1 << 31),
    dict(n_kv_heads=0), dict(n_kv_heads=2000), dict(head_dim=96), dict(head_dim=512)])
def test_bad_caches(lib, bad):
    assert append(lib, cache(**bad)) == -1
    assert attn(lib, cache(**bad)) == -1


@pytest.mark.parametrize("bad", [
    dict(c=False), dict(k=None), dict(k=AT + 8), dict(v=None), dict(stride=120), dict(stride=132), dict(B=0), dict(B=1025),
    dict(N=0), dict(N=-5), dict(N=(1 << 24) + 1), dict(lens=None), dict(lens=AT + 1), dict(table=AT + 2), dict(mb=0),
    dict(mb=(1 << 24) + 1)])
def test_bad_appends(lib, bad):
    assert append(lib, **bad) == -1 and lib.fgm_last_error()


@pytest.mark.parametrize("bad", [
    dict(c=False), dict(q=None), dict(q=AT + 4), dict(stride=255), dict(stride=248), dict(B=0), dict(M=0), dict(M=9),
    dict(Hq=0), dict(Hq=3), dict(Hq=32, M=8, stride=2048), dict(lens=None), dict(mb=0), dict(scale=0.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.0), dict(window=-1), dict(out=None),
    dict(out=AT + 2), dict(lse=AT + 2)])
def test_bad_attention_calls(lib, bad):
    assert attn(lib, **bad) == -1 and lib.fgm_last_error()


def test_bad_workspaces(lib):
    for call in (append, attn):
        assert call(lib, ws=None) == -2
        assert call(lib, ws=AT + 16) == -2
        assert call(lib, nws=1024) == -2
        assert b"needed" in lib.fgm_last_error()


def test_attn_workspace_bytes(lib):
    f = fgm.attn_workspace_bytes
    assert f(1, 5, 16, 8, 256) >= fgm.workspace_bytes(8) and f(1, 5, 16, 8, 256) % 256 == 0
    for bad in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 9, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 1, 1, 80), (1, 8, 9, 1, 64),
                (1, 1, 4, 0, 64), (1025, 1, 1, 1, 64)):
        assert f(*bad) == 0


def test_binding_refuses_host_tensors():
    c = fgm.KVCache.empty(2, 1, 64, device="cpu")
    with pytest.raises(fgm.FgmError):
        fgm.kv_append(c, torch.zeros(1, 1, 1, 64).bfloat16(), torch.zeros(1, 1, 1, 64).bfloat16(),
                      torch.ones(1, dtype=torch.int32))
    with pytest.raises(fgm.FgmError):
        fgm.attn_fwd(c, torch.zeros(1, 1, 1, 64).bfloat16(), torch.ones(1, dtype=torch.int32), 1.0)
