"""Host-side refusals of the routing, grouped products, experts and block norms:
nothing here reaches a GPU. And the order in which their kernels take tensor memory."""

import ctypes
import os
import re

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
BIG = 1 << 50


def route(lib, w=AT, b=AT, x=AT, stride=2816, T=4, ids=AT, wt=AT, off=AT, order=AT, ws=AT, nws=BIG):
    return lib.fgm_moe_route(w, b, x, stride, T, ids, wt, off, order, ws, nws, None)


@pytest.mark.parametrize("bad", [
    dict(w=None), dict(w=AT + 8), dict(b=AT + 2), dict(x=None), dict(x=AT + 2), dict(stride=2815), dict(stride=2808), dict(stride=2820),
    dict(stride=1 << 40), dict(T=0), dict(T=-1), dict(T=(1 << 18) + 1), dict(ids=None), dict(ids=AT + 1), dict(wt=None), dict(wt=AT + 2),
    dict(off=None), dict(order=None), dict(off=AT + 2), dict(order=AT + 2)])
def test_bad_routes(lib, bad):
    assert route(lib, **bad) == -1 and lib.fgm_last_error()


def group(lib, ids=AT, n=8, E=4, off=AT, order=AT, ws=AT, nws=BIG):
    return lib.fgm_moe_group(ids, n, E, off, order, ws, nws, None)


@pytest.mark.parametrize("bad", [
    dict(ids=None), dict(ids=AT + 2), dict(n=0), dict(n=(1 << 21) + 1), dict(E=0), dict(E=1025), dict(off=None), dict(off=AT + 1),
    dict(order=None), dict(order=AT + 2)])
def test_bad_groups(lib, bad):
    assert group(lib, **bad) == -1 and lib.fgm_last_error()


def gemm(lib, x=AT, stride=64, xr=5, rows=AT, per=2, off=AT, w=AT, wt=3, s=AT, E=3, N=10, K=64, out=AT, R=7, ws=AT, nws=BIG):
    return lib.fgm_grouped_gemm(x, stride, xr, rows, per, off, w, wt, s, E, N, K, out, R, ws, nws, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=AT + 8), dict(stride=63), dict(stride=56), dict(stride=68), dict(xr=0), dict(xr=(1 << 24) + 1), dict(rows=AT + 2),
    dict(rows=None), dict(per=0), dict(per=-3), dict(off=None), dict(off=AT + 2), dict(w=None), dict(w=AT + 8), dict(wt=0), dict(wt=2),
    dict(wt=4), dict(s=AT + 2), dict(E=0), dict(E=1025), dict(N=0), dict(N=65537), dict(K=0), dict(K=8), dict(K=24), dict(K=20, wt=1),
    dict(K=65544, stride=65544), dict(out=None), dict(out=AT + 1), dict(R=0), dict(R=(1 << 24) + 1)])
def test_bad_gemms(lib, bad):
    assert gemm(lib, **bad) == -1 and lib.fgm_last_error()


def layer(**kw):
    f = dict(router_w=None, router_b=None, gate_q=AT, gate_s=AT, up_q=AT, up_s=AT, down_q=AT, down_s=AT)
    f.update(kw)
    return fgm.fgm_layer(*[f[n] for n in ("router_w", "router_b", "gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s")])


def experts(lib, L=None, x=AT, stride=2816, T=4, ids=AT, w=AT, shared=1, y=AT, ws=AT, nws=BIG):
    return lib.fgm_moe_experts_fwd(None if L is False else ctypes.byref(L or layer()), x, stride, T, ids, w, shared, y, ws, nws, None)


@pytest.mark.parametrize("bad", [
    dict(L=False), dict(L=layer(gate_q=None)), dict(L=layer(up_q=AT + 8)), dict(L=layer(down_q=None)), dict(L=layer(gate_s=None)),
    dict(L=layer(up_s=AT + 2)), dict(L=layer(down_s=None)), dict(x=None), dict(x=AT + 8), dict(stride=2800), dict(stride=2817), dict(T=0),
    dict(T=(1 << 18) + 1), dict(ids=None), dict(ids=AT + 1), dict(w=None), dict(w=AT + 2), dict(y=None), dict(y=AT + 8)])
def test_bad_experts(lib, bad):
    assert experts(lib, **bad) == -1 and lib.fgm_last_error()


def test_bad_workspaces(lib):
    for call in (route, gemm, experts):
        assert call(lib, ws=None) == -2 and call(lib, ws=AT + 16) == -2 and call(lib, nws=4096) == -2
        assert b"needed" in lib.fgm_last_error()
    assert group(lib, ws=None) == -2 and group(lib, nws=64) == -2


def test_workspace_bytes():
    f, base = fgm, fgm.workspace_bytes(8)
    for n in (f.moe_route_workspace_bytes(5), f.moe_group_workspace_bytes(40, 128), f.grouped_gemm_workspace_bytes(5, 40, 8, 64, 64),
              f.moe_experts_workspace_bytes(1)):
        assert n >= base and n % 256 == 0
    assert f.moe_route_workspace_bytes(0) == f.moe_route_workspace_bytes((1 << 18) + 1) == 0
    assert f.moe_group_workspace_bytes(0, 8) == f.moe_group_workspace_bytes(8, 0) == f.moe_group_workspace_bytes(8, 1025) == 0
    for bad in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 1, 0, 1, 64), (1, 1, 1, 0, 64), (1, 1, 1, 1, 4), (1, 1, 1, 1, 12)):
        assert f.grouped_gemm_workspace_bytes(*bad) == 0
    assert f.moe_experts_workspace_bytes(0) == f.moe_experts_workspace_bytes((1 << 18) + 1) == 0


def block(**kw):
    f = dict(N=4, D=64, h_type=1, y_type=1, gate_type=1, gain_type=0, xn_type=1, h=AT, y=AT + 1024, gate=AT + 2048, post_gain=AT + 2560,
             pre_gain=AT + 2816, h_out=AT, xn=AT + 4096, h_stride=64, y_stride=64, gate_row_stride=64, h_out_stride=64, xn_stride=64,
             gate_col_stride=1, post_norm=1, residual_scale=1.0, block_scale=1.0, gain_offset=0.0, eps=1e-6)
    f.update(kw)
    return fgm.fgm_block(**f)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [
    dict(N=0), dict(N=1 << 31), dict(D=0), dict(D=16385, h_stride=20000, y_stride=20000, h_out_stride=20000, xn_stride=20000, gate_row_stride=20000),
    dict(h=None), dict(h=AT + 1), dict(h_type=3), dict(h_type=-1), dict(h_stride=63), dict(h_stride=1 << 40), dict(y=AT + 1025), dict(y_type=7),
    dict(y_stride=10), dict(y=None), dict(y=None, gate=None), dict(gate_type=5), dict(gate=AT + 2049), dict(gate_row_stride=63),
    dict(gate_row_stride=-64), dict(gate_col_stride=2), dict(gate_col_stride=-1), dict(gain_type=4), dict(post_gain=AT + 2562),
    dict(post_norm=0), dict(xn=None), dict(h_out=None, xn=None, pre_gain=None), dict(xn_type=3), dict(xn=AT + 4097), dict(xn_stride=1),
    dict(h_out_stride=0), dict(residual_scale=NAN), dict(block_scale=INF), dict(gain_offset=NAN), dict(eps=-1e-6), dict(eps=INF),
    # outputs over other tensors
    dict(h_out=AT + 2), dict(h_out=AT, h_out_stride=72), dict(xn=AT + 2), dict(xn=AT), dict(xn=AT + 64), dict(xn=AT + 1024, xn_type=0),
    dict(xn=AT + 1024, xn_stride=128), dict(xn=AT + 1026), dict(xn=AT + 2048), dict(xn=AT + 2560), dict(h_out=AT + 1024), dict(h_out=AT + 2048)])
def test_bad_blocks(lib, bad):
    assert lib.fgm_block_norm(ctypes.byref(block(**bad)), None) == -1 and lib.fgm_last_error()


@pytest.mark.parametrize("good", [
    dict(), dict(h_out=AT + 5120), dict(xn=AT + 1024), dict(xn=AT, h_out=None), dict(y=None, gate=None, post_gain=None),
    dict(xn=None, pre_gain=None), dict(gate=None), dict(gate_col_stride=0, gate_row_stride=1), dict(gate_row_stride=0),
    # halves of one tensor's rows
    dict(h=AT, h_stride=128, h_out=AT + 128, h_out_stride=128, N=4)])
def test_blocks_pass_the_checks(lib, good):
    """What is allowed is refused here for want of a GPU alone (with one, host addresses must not get that far)."""
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    assert lib.fgm_block_norm(ctypes.byref(block(**good)), None) in (-3, -4), lib.fgm_last_error()


def test_null_block(lib):
    assert lib.fgm_block_norm(None, None) == -1


def test_binding_refuses_host_tensors():
    x, ids = torch.zeros(2, 2816, dtype=torch.bfloat16), torch.zeros(2, 8, dtype=torch.int32)
    for call in (lambda: fgm.moe_route(torch.zeros(128, 2816, dtype=torch.bfloat16), x), lambda: fgm.moe_group(ids, 4),
                 lambda: fgm.grouped_gemm(x, torch.zeros(1, 8, 2816, dtype=torch.bfloat16), None, torch.zeros(2, dtype=torch.int32)),
                 lambda: fgm.block_norm(x)):
        with pytest.raises(fgm.FgmError):
            call()


def test_tensor_memory_is_taken_behind_the_wait():
    """A kernel that holds tensor memory while it waits for the one before it to end
    would hang with one that lets it start before taking its own."""
    csrc, found = os.path.join(os.path.dirname(fgm.__file__), "csrc"), 0
    for f in sorted(os.listdir(csrc)):
        code = re.sub(r"//[^\n]*", "", open(os.path.join(csrc, f)).read())
        for kernel in code.split("__global__")[1:]:
            if "memory_take<" in kernel:
                found += 1
                assert kernel.index("after_previous()") < kernel.index("memory_take<") < kernel.index("let_next_start()"), f
    assert found == 2
