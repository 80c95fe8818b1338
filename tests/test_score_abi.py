"""Host-side refusals of the log-probability entry points: nothing here reaches a GPU."""

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


def call(lib, z=AT, dtype=0, stride=100, N=2, V=100, T=1.0, tokens=AT, k=4, logp=AT, entropy=AT, ids=AT, tlp=AT, ws=AT,
         nws=1 << 40):
    return lib.fgm_logprobs(z, dtype, stride, N, V, T, tokens, k, logp, entropy, ids, tlp, ws, nws, None)


@pytest.mark.parametrize("bad", [
    dict(z=None), dict(z=AT + 2), dict(z=AT + 1, dtype=1), dict(dtype=3), dict(dtype=-1), dict(stride=99), dict(stride=1 << 41),
    dict(N=0), dict(N=(1 << 24) + 1), dict(V=0), dict(V=1 << 31, stride=1 << 31), dict(T=0.0), dict(T=-2.0), dict(T=float("nan")),
    dict(T=float("inf")), dict(T=1e-39), dict(tokens=None), dict(tokens=AT + 1), dict(k=-1), dict(k=17), dict(V=3, k=4),
    dict(ids=None), dict(tlp=None), dict(ids=AT + 2), dict(logp=AT + 2), dict(entropy=AT + 1)])
def test_bad_calls(lib, bad):
    assert call(lib, **bad) == -1 and lib.fgm_last_error()


def lm(lib, emb=AT, V=100, h=AT, N=2, T=1.0, tokens=AT, k=4, logp=AT, entropy=AT, ids=AT, tlp=AT, ws=AT, nws=1 << 40):
    return lib.fgm_lm_head_logprobs(emb, V, h, N, T, tokens, k, logp, entropy, ids, tlp, ws, nws, None)


@pytest.mark.parametrize("bad", [
    dict(emb=None), dict(emb=AT + 8), dict(h=None), dict(h=AT + 2), dict(N=0), dict(N=(1 << 24) + 1), dict(V=0), dict(V=1 << 31),
    dict(T=0.0), dict(T=float("nan")), dict(tokens=None), dict(k=-1), dict(k=17), dict(V=3, k=4), dict(ids=None),
    dict(tlp=AT + 2)])
def test_bad_lm_head_calls(lib, bad):
    assert lm(lib, **bad) == -1 and lib.fgm_last_error()


def test_bad_workspaces(lib):
    assert lm(lib, ws=None) == -2 and lm(lib, ws=AT + 16) == -2 and lm(lib, nws=1024) == -2
    assert fgm.lm_head_logprobs_workspace_bytes(5, 262144, 8) > fgm.workspace_bytes(8)
    assert fgm.lm_head_logprobs_workspace_bytes(0, 10, 1) == 0

    assert call(lib, ws=None) == -2
    assert call(lib, ws=AT + 16) == -2
    assert call(lib, nws=1024) == -2


def test_workspace_bytes(lib):
    f = fgm.logprobs_workspace_bytes
    assert f(5, 262144, 8) > fgm.workspace_bytes(8) and f(5, 262144, 8) % 256 == 0
    assert f(1 << 20, 100, 0) >= fgm.workspace_bytes(8)
    for bad in ((0, 10, 1), (1, 0, 0), (1, 10, 11), (1, 100, 17), (1, 100, -1), (1, 1 << 31, 1), ((1 << 24) + 1, 10, 1)):
        assert f(*bad) == 0


def test_binding_refuses_host_tensors():
    with pytest.raises(fgm.FgmError):
        fgm.logprobs(torch.zeros(2, 5))
