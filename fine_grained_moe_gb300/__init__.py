"""Python binding of the GB300 batch-1 fine-grained MoE verify-step library.

A thin ctypes layer over the C ABI in ``include/fgm.h``: it turns torch CUDA
tensors into device pointers, picks the current CUDA stream and raises on a
non-zero status. Every stage of the step runs in the CUDA library
``libfgm.so``; there is no other implementation in this package, so calling
any function without the built library raises.

Build the library with ``python -m fine_grained_moe_gb300.build`` (or the
repository's ``__graft_entry__.build()``).
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import NamedTuple

import torch

from . import traffic  # noqa: F401  (byte accounting used by the benchmark)

HIDDEN = 2816
FFN = 704
EXPERTS = 128
N_EXPERTS = 129
TOPK = 8
MAX_M = 8
MAX_LAYERS = 48

STATUS_NONFINITE_LOGITS = 1
STATUS_WAIT_TIMEOUT = 2
STATUS_NONFINITE_KV = 4
STATUS_BAD_BLOCK = 8
MAX_TOKENS = 1 << 18  # tokens of moe_route and moe_experts_fwd
MAX_GROUPS = 1024  # experts of moe_group and grouped_gemm
E4M3 = 3           # element type of 8-bit weights in the C ABI
MAX_TOP = 16       # alternatives per row of the log-probability calls
KV_BLOCK = 64      # tokens of a KV-cache block
ATTN_MAX_ROWS = 64  # query rows sharing a kv head: M * n_q_heads / n_kv_heads
PATH_FUSED = 0    # one persistent cooperative kernel per call (TMA ring + mma.sync tiles; tcgen05 down products at M <= 5)
PATH_STAGED = 1   # one launch per stage, fp32 CUDA-core arithmetic
PATH_FUSED_TC = 2  # as PATH_FUSED, with the FP8 lm_head on tcgen05 tensor-memory tiles fed by TMA tensor copies
PATH_FUSED_MMA = 3  # as PATH_FUSED, with the down products on mma.sync at every M (comparison path)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfgm.so")
_lib = None


class FgmError(RuntimeError):
    pass


class fgm_layer(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("router_w", "router_b", "gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s")]


class fgm_mlp(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s")] + \
               [("width", ctypes.c_int)]


class fgm_kv_cache(ctypes.Structure):
    _fields_ = [("k_q", ctypes.c_void_p), ("k_s", ctypes.c_void_p), ("v_q", ctypes.c_void_p), ("v_s", ctypes.c_void_p),
                ("n_blocks", ctypes.c_int64), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class fgm_block(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("D", ctypes.c_int)] + \
               [(n, ctypes.c_int) for n in ("h_type", "y_type", "gate_type", "gain_type", "xn_type")] + \
               [(n, ctypes.c_void_p) for n in ("h", "y", "gate", "post_gain", "pre_gain", "h_out", "xn")] + \
               [(n, ctypes.c_int64) for n in ("h_stride", "y_stride", "gate_row_stride", "h_out_stride", "xn_stride")] + \
               [("gate_col_stride", ctypes.c_int), ("post_norm", ctypes.c_int)] + \
               [(n, ctypes.c_float) for n in ("residual_scale", "block_scale", "gain_offset", "eps")]


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise FgmError(f"CUDA library not built: {LIB_PATH} is missing "
                           "(run python -m fine_grained_moe_gb300.build)")
        L = ctypes.CDLL(LIB_PATH)
        vp, ci, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        LP = ctypes.POINTER(fgm_layer)
        CP = ctypes.POINTER(fgm_kv_cache)
        sig = {
            "fgm_workspace_bytes": (sz, [ci, i64]),
            "fgm_workspace_init": (ci, [vp, sz, vp]),
            "fgm_moe_layer_fwd": (ci, [LP, vp, vp, ci, vp, vp, vp, sz, vp]),
            "fgm_moe_layer_fwd_noalloc": (ci, [LP, vp, vp, ci, vp, vp, vp]),
            "fgm_moe_stack_fwd": (ci, [LP, ci, vp, vp, ci, vp, vp, sz, vp]),
            "fgm_moe_layer_dense_fwd": (ci, [LP, ctypes.POINTER(fgm_mlp), vp, vp, ci, vp, vp, vp, sz, vp]),
            "fgm_moe_stack_dense_fwd": (ci, [LP, ctypes.POINTER(fgm_mlp), ci, vp, vp, ci, vp, vp, sz, vp]),
            "fgm_verify_step_dense": (ci, [LP, ctypes.POINTER(fgm_mlp), ci, vp, i64, vp, vp, ci, vp, vp, vp, sz,
                                           vp]),
            "fgm_lm_head_argmax": (ci, [vp, i64, vp, ci, vp, vp, vp, sz, vp]),
            "fgm_lm_head_argmax_fp8": (ci, [vp, vp, i64, vp, ci, vp, vp, vp, sz, vp]),
            "fgm_spec_verify": (ci, [vp, vp, ci, vp, vp]),
            "fgm_verify_step": (ci, [LP, ci, vp, i64, vp, vp, ci, vp, vp, vp, sz, vp]),
            "fgm_verify_step_host": (ci, [LP, ci, vp, i64, vp, vp, ci, vp, vp, sz, vp]),
            "fgm_verify_step_fp8_head": (ci, [LP, ci, vp, vp, i64, vp, vp, ci, vp, vp, vp, sz, vp]),
            "fgm_lm_head_sample": (ci, [vp, i64, vp, ci, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "fgm_verify_step_sample": (ci, [LP, ci, vp, i64, vp, vp, ci, ctypes.c_float, vp, vp, vp, vp, vp, vp,
                                            sz, vp]),
            "fgm_kv_append": (ci, [CP, vp, vp, i64, ci, ci, vp, vp, ci, vp, sz, vp]),
            "fgm_attn_workspace_bytes": (sz, [ci, ci, ci, ci, ci]),
            "fgm_attn_fwd": (ci, [CP, vp, i64, ci, ci, ci, vp, vp, ci, ctypes.c_float, ci, vp, vp, vp, sz, vp]),
            "fgm_logprobs_workspace_bytes": (sz, [i64, i64, ci]),
            "fgm_logprobs": (ci, [vp, ci, i64, i64, i64, ctypes.c_float, vp, ci, vp, vp, vp, vp, vp, sz, vp]),
            "fgm_lm_head_logprobs_workspace_bytes": (sz, [i64, i64, ci]),
            "fgm_lm_head_logprobs": (ci, [vp, i64, vp, i64, ctypes.c_float, vp, ci, vp, vp, vp, vp, vp, sz, vp]),
            "fgm_moe_route_workspace_bytes": (sz, [i64]),
            "fgm_moe_route": (ci, [vp, vp, vp, i64, i64, vp, vp, vp, vp, vp, sz, vp]),
            "fgm_moe_group_workspace_bytes": (sz, [i64, ci]),
            "fgm_moe_group": (ci, [vp, i64, ci, vp, vp, vp, sz, vp]),
            "fgm_grouped_gemm_workspace_bytes": (sz, [i64, i64, ci, ci, ci]),
            "fgm_grouped_gemm": (ci, [vp, i64, i64, vp, ci, vp, vp, ci, vp, ci, ci, ci, vp, i64, vp, sz, vp]),
            "fgm_moe_experts_workspace_bytes": (sz, [i64]),
            "fgm_moe_experts_fwd": (ci, [LP, vp, i64, i64, vp, vp, ci, vp, vp, sz, vp]),
            "fgm_block_norm": (ci, [ctypes.POINTER(fgm_block), vp]),
            "fgm_read_status": (ci, [vp, sz, ci, vp, vp]),
            "fgm_select_path": (ci, [ci]),
            "fgm_set_phase_trace": (ci, [vp, sz]),
            "fgm_debug_stall_next_launch": (ci, []),
            "fgm_debug_stall_next_launch_at": (ci, [ci]),
            "fgm_read_wait_report": (ci, [vp, sz, vp, vp]),
            "fgm_set_wait_limit_ns": (ctypes.c_longlong, [ctypes.c_longlong]),
            "fgm_last_error": (ctypes.c_char_p, []),
            "fgm_version": (ci, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(rc: int) -> None:
    if rc != 0:
        msg = lib().fgm_last_error().decode(errors="replace")
        raise FgmError(f"fgm error {rc}: {msg}")


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise FgmError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise FgmError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _m(x: torch.Tensor) -> int:
    if x.dim() != 2 or x.shape[1] != HIDDEN or x.dtype != torch.bfloat16:
        raise FgmError(f"expected bf16 [M, {HIDDEN}] activations, got {tuple(x.shape)} {x.dtype}")
    return int(x.shape[0])


def _check_like(name: str, t: torch.Tensor, x: torch.Tensor) -> None:
    """Output rows must match the input rows: bf16 [M, 2816] on x's device."""
    if tuple(t.shape) != tuple(x.shape) or t.dtype != torch.bfloat16 or t.device != x.device:
        raise FgmError(f"{name}: expected bf16 {tuple(x.shape)} on {x.device}, got "
                       f"{tuple(t.shape)} {t.dtype} on {t.device}")


def _check_topk(M: int, x: torch.Tensor, topk_ids: torch.Tensor | None, topk_w: torch.Tensor | None) -> None:
    """Optional routing outputs: int32 / float32 [M, 8] on x's device."""
    for name, t, dt in (("topk_ids", topk_ids, torch.int32), ("topk_w", topk_w, torch.float32)):
        if t is not None and (tuple(t.shape) != (M, TOPK) or t.dtype != dt or t.device != x.device):
            raise FgmError(f"{name}: expected {dt} [{M}, {TOPK}] on {x.device}, got "
                           f"{tuple(t.shape)} {t.dtype} on {t.device}")


def select_path(path: int) -> int:
    """Selects the execution path (PATH_FUSED, PATH_STAGED, PATH_FUSED_TC or PATH_FUSED_MMA); returns the previous one."""
    return int(lib().fgm_select_path(int(path)))


def set_wait_limit_ns(ns: int) -> int:
    """Bound on every wait inside the persistent kernel, attn_fwd's, lm_head_logprobs', moe_route's, grouped_gemm's and
    moe_experts_fwd's (ns < 0 only queries)."""
    return int(lib().fgm_set_wait_limit_ns(int(ns)))


def set_phase_trace(buf: torch.Tensor | None) -> None:
    """Profiling aid: record per-CTA phase timestamps of later persistent-kernel
    launches into an int64 CUDA tensor (None stops)."""
    if buf is None:
        _check(lib().fgm_set_phase_trace(None, 0))
    else:
        if buf.dtype != torch.int64:
            raise FgmError("trace buffer must be int64")
        _check(lib().fgm_set_phase_trace(_ptr(buf), buf.numel()))


def debug_stall_next_launch(layer: int = 0) -> None:
    """Test hook: the next persistent-kernel launch waits, at the start of
    ``layer``, on a barrier that can never complete, so its wait limit must run
    out."""
    if layer == 0:
        _check(lib().fgm_debug_stall_next_launch())
    else:
        _check(lib().fgm_debug_stall_next_launch_at(int(layer)))


def workspace_bytes(M: int = MAX_M, V: int = 0) -> int:
    return int(lib().fgm_workspace_bytes(int(M), int(V)))


class Workspace:
    """Device scratch for the library's calls (one per concurrent stream).
    ``nbytes`` raises its size to what a call's own ``*_workspace_bytes`` says."""

    def __init__(self, device=None, M: int = MAX_M, V: int = 0, nbytes: int = 0):
        self.nbytes = max(workspace_bytes(M, V), int(nbytes))
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device or "cuda")
        off = (-self.buf.data_ptr()) % 256
        self.t = self.buf[off:off + self.nbytes]
        _check(lib().fgm_workspace_init(_ptr(self.t), self.nbytes, _stream(None)))

    @property
    def ptr(self):
        return _ptr(self.t)

    def wait_report(self) -> list[int]:
        """{site, block, warp, index} of the first wait that ran out (see fgm.h)."""
        out = (ctypes.c_int32 * 4)()
        _check(lib().fgm_read_wait_report(self.ptr, self.nbytes, out, _stream(None)))
        return list(out)

    def status(self, clear: bool = True) -> int:
        out = ctypes.c_int32(0)
        _check(lib().fgm_read_status(self.ptr, self.nbytes, int(clear), ctypes.byref(out), _stream(None)))
        return int(out.value)


@dataclass
class Layer:
    """One layer's device tensors (see ``fgm_layer`` in include/fgm.h)."""
    router_w: torch.Tensor
    router_b: torch.Tensor | None
    gate_q: torch.Tensor
    gate_s: torch.Tensor
    up_q: torch.Tensor
    up_s: torch.Tensor
    down_q: torch.Tensor
    down_s: torch.Tensor

    @classmethod
    def from_dict(cls, p: dict) -> "Layer":
        return cls(**{k: p[k] for k in ("router_w", "router_b", "gate_q", "gate_s", "up_q", "up_s",
                                        "down_q", "down_s")})

    def struct(self) -> fgm_layer:
        shapes = {"router_w": ((EXPERTS, HIDDEN), torch.bfloat16),
                  "gate_q": ((N_EXPERTS, FFN, HIDDEN), torch.uint8),
                  "up_q": ((N_EXPERTS, FFN, HIDDEN), torch.uint8),
                  "down_q": ((N_EXPERTS, HIDDEN, FFN), torch.uint8),
                  "gate_s": ((N_EXPERTS, FFN), torch.float32),
                  "up_s": ((N_EXPERTS, FFN), torch.float32),
                  "down_s": ((N_EXPERTS, HIDDEN), torch.float32)}
        for name, (shape, dt) in shapes.items():
            t = getattr(self, name)
            if tuple(t.shape) != shape or t.dtype != dt:
                raise FgmError(f"{name}: expected {shape} {dt}, got {tuple(t.shape)} {t.dtype}")
        if self.router_b is not None and (tuple(self.router_b.shape) != (EXPERTS,)
                                          or self.router_b.dtype != torch.float32):
            raise FgmError("router_b: expected float32 [128]")
        return fgm_layer(*[(_ptr(getattr(self, n)) or ctypes.c_void_p(0)).value for n in
                           ("router_w", "router_b", "gate_q", "gate_s", "up_q", "up_s", "down_q",
                            "down_s")])


def _layers_array(layers) -> ctypes.Array:
    structs = [(l if isinstance(l, Layer) else Layer.from_dict(l)).struct() for l in layers]
    arr = (fgm_layer * len(structs))(*structs)
    return arr


def _ws(ws: Workspace | None, device) -> Workspace:
    return ws if ws is not None else Workspace(device)


# ---------------------------------------------------------------- entry points
def moe_layer_fwd(layer, x: torch.Tensor, y: torch.Tensor | None = None,
                  topk_ids: torch.Tensor | None = None, topk_w: torch.Tensor | None = None,
                  ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """One MoE layer (no norm, no residual) on bf16 x[M, 2816]; returns bf16 y."""
    M = _m(x)
    y = torch.empty_like(x) if y is None else y
    _check_like("y", y, x)
    _check_topk(M, x, topk_ids, topk_w)
    ws = _ws(ws, x.device)
    L = (layer if isinstance(layer, Layer) else Layer.from_dict(layer)).struct()
    _check(lib().fgm_moe_layer_fwd(ctypes.byref(L), _ptr(x), _ptr(y), M, _ptr(topk_ids), _ptr(topk_w),
                                   ws.ptr, ws.nbytes, _stream(stream)))
    return y


def _mlp_struct(mlp: dict) -> fgm_mlp:
    W = int(mlp["gate_q"].shape[0])
    shapes = {"gate_q": ((W, HIDDEN), torch.uint8), "up_q": ((W, HIDDEN), torch.uint8),
              "down_q": ((HIDDEN, W), torch.uint8), "gate_s": ((W,), torch.float32),
              "up_s": ((W,), torch.float32), "down_s": ((HIDDEN,), torch.float32)}
    for name, (shape, dt) in shapes.items():
        t = mlp[name]
        if tuple(t.shape) != shape or t.dtype != dt or not t.is_contiguous():
            raise FgmError(f"dense {name}: expected contiguous {shape} {dt}, got {tuple(t.shape)} {t.dtype}")
    return fgm_mlp(*[_ptr(mlp[n]).value for n in ("gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s")],
                   W)


def moe_layer_dense_fwd(layer, dense: dict, x: torch.Tensor, y: torch.Tensor | None = None,
                        topk_ids: torch.Tensor | None = None, topk_w: torch.Tensor | None = None,
                        ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """One MoE layer with the always-on dense MLP `dense` (gate_q/up_q [W, 2816],
    down_q [2816, W], fp32 row scales; W a multiple of 704 up to 2112) in place
    of the shared expert; returns bf16 y."""
    M = _m(x)
    y = torch.empty_like(x) if y is None else y
    _check_like("y", y, x)
    _check_topk(M, x, topk_ids, topk_w)
    ws = _ws(ws, x.device)
    L = (layer if isinstance(layer, Layer) else Layer.from_dict(layer)).struct()
    D = _mlp_struct(dense)
    _check(lib().fgm_moe_layer_dense_fwd(ctypes.byref(L), ctypes.byref(D), _ptr(x), _ptr(y), M, _ptr(topk_ids),
                                         _ptr(topk_w), ws.ptr, ws.nbytes, _stream(stream)))
    return y


def moe_layer_fwd_noalloc(layer, x: torch.Tensor, y: torch.Tensor,
                          topk_ids: torch.Tensor | None = None, topk_w: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """moe_layer_fwd on the library's built-in device scratch instead of a
    Workspace, for callers that must not allocate while they run (``y`` is
    therefore required). At most 8 tokens. Calls whose GPU work overlaps on
    one device race on that scratch; make the first call on a device before
    any stream capture starts, since it looks the scratch up."""
    M = _m(x)
    _check_like("y", y, x)
    _check_topk(M, x, topk_ids, topk_w)
    L = (layer if isinstance(layer, Layer) else Layer.from_dict(layer)).struct()
    _check(lib().fgm_moe_layer_fwd_noalloc(ctypes.byref(L), _ptr(x), _ptr(y), M, _ptr(topk_ids),
                                           _ptr(topk_w), _stream(stream)))
    return y


def moe_stack_fwd(layers, x: torch.Tensor, y: torch.Tensor | None = None,
                  ids_trace: torch.Tensor | None = None, ws: Workspace | None = None,
                  stream=None) -> torch.Tensor:
    """The stack h <- h + layer(RMSNorm(h)) over ``layers``; returns bf16 h."""
    M = _m(x)
    y = torch.empty_like(x) if y is None else y
    _check_like("y", y, x)
    if ids_trace is not None and (tuple(ids_trace.shape) != (len(layers), M, TOPK)
                                  or ids_trace.dtype != torch.int32 or ids_trace.device != x.device):
        raise FgmError(f"ids_trace: expected int32 [{len(layers)}, {M}, {TOPK}] on {x.device}")
    ws = _ws(ws, x.device)
    arr = _layers_array(layers)
    _check(lib().fgm_moe_stack_fwd(arr, len(arr), _ptr(x), _ptr(y), M, _ptr(ids_trace), ws.ptr,
                                   ws.nbytes, _stream(stream)))
    return y


def _mlps_array(mlps, n_layers: int) -> ctypes.Array:
    if len(mlps) != n_layers:
        raise FgmError(f"mlps: expected one dense MLP per layer ({n_layers}), got {len(mlps)}")
    return (fgm_mlp * n_layers)(*[_mlp_struct(m) for m in mlps])


def moe_stack_dense_fwd(layers, mlps, x: torch.Tensor, y: torch.Tensor | None = None,
                        ids_trace: torch.Tensor | None = None, ws: Workspace | None = None,
                        stream=None) -> torch.Tensor:
    """The stack with the dense MLP ``mlps[l]`` (dicts as for moe_layer_dense_fwd)
    in place of layer l's shared expert; returns bf16 h."""
    M = _m(x)
    y = torch.empty_like(x) if y is None else y
    _check_like("y", y, x)
    if ids_trace is not None and (tuple(ids_trace.shape) != (len(layers), M, TOPK)
                                  or ids_trace.dtype != torch.int32 or ids_trace.device != x.device):
        raise FgmError(f"ids_trace: expected int32 [{len(layers)}, {M}, {TOPK}] on {x.device}")
    ws = _ws(ws, x.device)
    arr = _layers_array(layers)
    mlp_arr = _mlps_array(mlps, len(arr))
    _check(lib().fgm_moe_stack_dense_fwd(arr, mlp_arr, len(arr), _ptr(x), _ptr(y), M, _ptr(ids_trace), ws.ptr,
                                         ws.nbytes, _stream(stream)))
    return y


def lm_head_argmax(emb: torch.Tensor, h: torch.Tensor, argmax: torch.Tensor | None = None,
                   maxlogit: torch.Tensor | None = None, ws: Workspace | None = None,
                   stream=None) -> torch.Tensor:
    """argmax_v emb[v] . h[t] for each of the M rows of bf16 h; returns int32 [M]."""
    M = _m(h)
    V = int(emb.shape[0])
    argmax = torch.empty(M, dtype=torch.int32, device=h.device) if argmax is None else argmax
    ws = _ws(ws, h.device)
    _check(lib().fgm_lm_head_argmax(_ptr(emb), V, _ptr(h), M, _ptr(argmax), _ptr(maxlogit), ws.ptr,
                                    ws.nbytes, _stream(stream)))
    return argmax


def _fp8_rows(emb_q: torch.Tensor, emb_s: torch.Tensor) -> int:
    if emb_q.dim() != 2 or emb_q.shape[1] != HIDDEN or emb_q.dtype != torch.uint8:
        raise FgmError(f"expected uint8 [V, {HIDDEN}] E4M3 codes, got {tuple(emb_q.shape)} {emb_q.dtype}")
    if emb_s.dtype != torch.float32 or tuple(emb_s.shape) != (emb_q.shape[0],):
        raise FgmError(f"expected fp32 [{emb_q.shape[0]}] row scales, got {tuple(emb_s.shape)} {emb_s.dtype}")
    return int(emb_q.shape[0])


def lm_head_argmax_fp8(emb_q: torch.Tensor, emb_s: torch.Tensor, h: torch.Tensor,
                       argmax: torch.Tensor | None = None, maxlogit: torch.Tensor | None = None,
                       ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """argmax_v emb_s[v] * (e4m3(emb_q[v]) . h[t]) for each of the M rows of bf16 h;
    returns int32 [M]."""
    M = _m(h)
    V = _fp8_rows(emb_q, emb_s)
    argmax = torch.empty(M, dtype=torch.int32, device=h.device) if argmax is None else argmax
    ws = _ws(ws, h.device)
    _check(lib().fgm_lm_head_argmax_fp8(_ptr(emb_q), _ptr(emb_s), V, _ptr(h), M, _ptr(argmax),
                                        _ptr(maxlogit), ws.ptr, ws.nbytes, _stream(stream)))
    return argmax


def _sample_args(M: int, V: int, device, draft, u_acc, u_next, z, out):
    if u_next is None or u_next.dtype != torch.float32 or u_next.numel() != M:
        raise FgmError(f"u_next must be fp32 [{M}]")
    if M > 1 and (draft is None or u_acc is None or u_acc.dtype != torch.float32 or u_acc.numel() != M - 1
                  or draft.dtype != torch.int32 or draft.numel() != M - 1):
        raise FgmError(f"draft (int32) and u_acc (fp32) must have M - 1 = {M - 1} elements")
    z = torch.empty((M, V), dtype=torch.float32, device=device) if z is None else z
    if z.dtype != torch.float32 or tuple(z.shape) != (M, V) or not z.is_contiguous():
        raise FgmError(f"z must be contiguous fp32 [{M}, {V}]")
    out = torch.empty(2, dtype=torch.int32, device=device) if out is None else out
    return z, out


def lm_head_sample(emb: torch.Tensor, h: torch.Tensor, T: float, draft: torch.Tensor | None,
                   u_acc: torch.Tensor | None, u_next: torch.Tensor, z: torch.Tensor | None = None,
                   argmax: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   ws: Workspace | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Speculative sampling verify at temperature T on the lm_head logits of the
    M bf16 rows h; returns (out int32 [2] = {accepted drafts, emitted token},
    z fp32 [M, V] logits)."""
    M = _m(h)
    V = int(emb.shape[0])
    z, out = _sample_args(M, V, h.device, draft, u_acc, u_next, z, out)
    ws = _ws(ws, h.device)
    _check(lib().fgm_lm_head_sample(_ptr(emb), V, _ptr(h), M, float(T), _ptr(draft) if M > 1 else None,
                                    _ptr(u_acc) if M > 1 else None, _ptr(u_next), _ptr(z), _ptr(argmax),
                                    _ptr(out), ws.ptr, ws.nbytes, _stream(stream)))
    return out, z


def verify_step_sample(layers, emb: torch.Tensor, x: torch.Tensor, T: float, draft: torch.Tensor | None,
                       u_acc: torch.Tensor | None, u_next: torch.Tensor, z: torch.Tensor | None = None,
                       argmax: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       ws: Workspace | None = None, stream=None, _arr=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Stack + final RMSNorm + lm_head + speculative sampling at temperature T;
    returns (out int32 [2] = {accepted drafts, emitted token}, z fp32 [M, V])."""
    M = _m(x)
    V = int(emb.shape[0])
    z, out = _sample_args(M, V, x.device, draft, u_acc, u_next, z, out)
    ws = _ws(ws, x.device)
    arr = _layers_array(layers) if _arr is None else _arr
    _check(lib().fgm_verify_step_sample(arr, len(arr), _ptr(emb), V, _ptr(x), _ptr(draft) if M > 1 else None, M,
                                        float(T), _ptr(u_acc) if M > 1 else None, _ptr(u_next), _ptr(z),
                                        _ptr(argmax), _ptr(out), ws.ptr, ws.nbytes, _stream(stream)))
    return out, z


def spec_verify(target: torch.Tensor, draft: torch.Tensor, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Greedy acceptance; returns int32 [2] = {accepted drafts, next token}."""
    M = int(target.shape[0])
    out = torch.empty(2, dtype=torch.int32, device=target.device) if out is None else out
    _check(lib().fgm_spec_verify(_ptr(target), _ptr(draft) if M > 1 else None, M, _ptr(out),
                                 _stream(stream)))
    return out


def verify_step(layers, emb: torch.Tensor, x: torch.Tensor, draft: torch.Tensor | None,
                out: torch.Tensor | None = None, argmax: torch.Tensor | None = None,
                ws: Workspace | None = None, stream=None, _arr=None) -> torch.Tensor:
    """Stack + final RMSNorm + lm_head argmax + greedy acceptance; returns int32
    [2] = {accepted drafts, next token} on the device."""
    M = _m(x)
    out = torch.empty(2, dtype=torch.int32, device=x.device) if out is None else out
    ws = _ws(ws, x.device)
    arr = _layers_array(layers) if _arr is None else _arr
    _check(lib().fgm_verify_step(arr, len(arr), _ptr(emb), int(emb.shape[0]), _ptr(x),
                                 _ptr(draft) if M > 1 else None, M, _ptr(argmax), _ptr(out), ws.ptr,
                                 ws.nbytes, _stream(stream)))
    return out


def verify_step_dense(layers, mlps, emb: torch.Tensor, x: torch.Tensor, draft: torch.Tensor | None,
                      out: torch.Tensor | None = None, argmax: torch.Tensor | None = None,
                      ws: Workspace | None = None, stream=None, _arr=None, _mlp_arr=None) -> torch.Tensor:
    """verify_step on the stack with a dense MLP per layer (see moe_stack_dense_fwd);
    returns int32 [2] = {accepted drafts, next token} on the device."""
    M = _m(x)
    out = torch.empty(2, dtype=torch.int32, device=x.device) if out is None else out
    ws = _ws(ws, x.device)
    arr = _layers_array(layers) if _arr is None else _arr
    mlp_arr = _mlps_array(mlps, len(arr)) if _mlp_arr is None else _mlp_arr
    _check(lib().fgm_verify_step_dense(arr, mlp_arr, len(arr), _ptr(emb), int(emb.shape[0]), _ptr(x),
                                       _ptr(draft) if M > 1 else None, M, _ptr(argmax), _ptr(out), ws.ptr,
                                       ws.nbytes, _stream(stream)))
    return out


def mlps_array(mlps):
    """Pre-marshalled dense MLP table, reusable across calls (pass as ``_mlp_arr``)."""
    return _mlps_array(mlps, len(mlps))


def verify_step_fp8_head(layers, emb_q: torch.Tensor, emb_s: torch.Tensor, x: torch.Tensor,
                         draft: torch.Tensor | None, out: torch.Tensor | None = None,
                         argmax: torch.Tensor | None = None, ws: Workspace | None = None, stream=None,
                         _arr=None) -> torch.Tensor:
    """verify_step with the FP8 lm_head (E4M3 rows emb_q, fp32 row scales emb_s);
    returns int32 [2] = {accepted drafts, next token} on the device."""
    M = _m(x)
    V = _fp8_rows(emb_q, emb_s)
    out = torch.empty(2, dtype=torch.int32, device=x.device) if out is None else out
    ws = _ws(ws, x.device)
    arr = _layers_array(layers) if _arr is None else _arr
    _check(lib().fgm_verify_step_fp8_head(arr, len(arr), _ptr(emb_q), _ptr(emb_s), V, _ptr(x),
                                          _ptr(draft) if M > 1 else None, M, _ptr(argmax), _ptr(out),
                                          ws.ptr, ws.nbytes, _stream(stream)))
    return out


def verify_step_host(layers, emb: torch.Tensor, x_host: torch.Tensor, draft_host: torch.Tensor | None,
                     out_host: torch.Tensor | None = None, ws: Workspace | None = None,
                     stream=None, _arr=None) -> torch.Tensor:
    """verify_step with host (ideally pinned) x/draft/out; synchronises."""
    if x_host.is_cuda:
        raise FgmError("x_host must be a host tensor")
    M = int(x_host.shape[0])
    out_host = torch.empty(2, dtype=torch.int32) if out_host is None else out_host
    ws = _ws(ws, emb.device)
    arr = _layers_array(layers) if _arr is None else _arr
    dp = ctypes.c_void_p(draft_host.data_ptr()) if (draft_host is not None and M > 1) else None
    _check(lib().fgm_verify_step_host(arr, len(arr), _ptr(emb), int(emb.shape[0]),
                                      ctypes.c_void_p(x_host.data_ptr()), dp, M,
                                      ctypes.c_void_p(out_host.data_ptr()), ws.ptr, ws.nbytes,
                                      _stream(stream)))
    return out_host


def layers_array(layers):
    """Pre-marshalled layer table, reusable across calls (pass as ``_arr``)."""
    return _layers_array(layers)


# ---------------------------------------------------------------- 8-bit KV cache
# (A call at a few microseconds of GPU time is bound by its host side: these
# wrappers check what they must with plain attribute reads, pass addresses as
# integers and enter a stream context only when the call names another stream
# or device than the current one.)
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _expect(name: str, t: torch.Tensor, shape: tuple, dtype, device) -> int:
    """Address of a contiguous tensor of this shape and type on ``device``."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise FgmError(f"{name}: expected {dtype} {tuple(shape)} on {device}, got {tuple(t.shape)} {t.dtype} on {t.device}")
    if not t.is_contiguous():
        raise FgmError(f"{name}: expected a contiguous tensor, strides {t.stride()}")
    return t.data_ptr()


@dataclass(frozen=True, eq=False)
class KVCache:
    """One layer's 8-bit cache (see ``fgm_kv_cache`` in include/fgm.h): E4M3
    codes k_q [blocks, kv heads, D / 64, 64, 64] and v_q [blocks, kv heads, D,
    64] as uint8, fp32 scales k_s, v_s [blocks, kv heads]."""
    k_q: torch.Tensor
    v_q: torch.Tensor
    k_s: torch.Tensor
    v_s: torch.Tensor

    @classmethod
    def empty(cls, n_blocks: int, n_kv_heads: int, head_dim: int, device="cuda") -> "KVCache":
        """A cache of n_blocks blocks of 64 tokens, not initialised: kv_append
        writes a block's scales with its first token."""
        if head_dim not in (64, 128, 256):
            raise FgmError(f"head_dim must be 64, 128 or 256, got {head_dim}")
        u8 = dict(dtype=torch.uint8, device=device)
        return cls(torch.empty((n_blocks, n_kv_heads, head_dim // 64, KV_BLOCK, 64), **u8),
                   torch.empty((n_blocks, n_kv_heads, head_dim, KV_BLOCK), **u8),
                   torch.empty((n_blocks, n_kv_heads), dtype=torch.float32, device=device),
                   torch.empty((n_blocks, n_kv_heads), dtype=torch.float32, device=device))

    @property
    def head_dim(self) -> int:
        return int(self.v_q.shape[2])

    @property
    def n_kv_heads(self) -> int:
        return int(self.v_q.shape[1])

    def struct(self) -> fgm_kv_cache:
        """The C struct of the four tensors, checked on its first use."""
        c = self.__dict__.get("_struct")
        if c is None:
            if self.v_q.dim() != 4 or self.v_q.shape[3] != KV_BLOCK:
                raise FgmError(f"v_q: expected [blocks, kv heads, D, {KV_BLOCK}], got {tuple(self.v_q.shape)}")
            if not self.v_q.is_cuda:
                raise FgmError("expected a CUDA tensor")
            n, h, d = (int(x) for x in self.v_q.shape[:3])
            dev = self.v_q.device
            c = fgm_kv_cache(_expect("k_q", self.k_q, (n, h, d // 64, KV_BLOCK, 64), _U8, dev),
                             _expect("k_s", self.k_s, (n, h), _F32, dev),
                             _expect("v_q", self.v_q, (n, h, d, KV_BLOCK), _U8, dev),
                             _expect("v_s", self.v_s, (n, h), _F32, dev), n, h, d)
            self.__dict__["_struct"] = c
        return c


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same in a tenth of the time, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _call(device: torch.device, stream, body):
    """Runs body(stream address) with ``device`` and the stream current, so that
    workspaces and outputs made inside belong to that stream."""
    if stream is None:
        if torch.cuda.current_device() == device.index:
            return body(_raw_stream(device.index))
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise FgmError(f"the stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def _space(ws: Workspace | None, device: torch.device, size=None, *args) -> Workspace:
    """The caller's workspace, or one of size(*args) bytes for this call."""
    if ws is None:
        return Workspace(device, nbytes=size(*args) if size else 0)
    if ws.t.device != device:
        raise FgmError(f"the workspace is on {ws.t.device}, the tensors on {device}")
    return ws


def _layer_on(layer, device: torch.device) -> fgm_layer:
    """A layer's struct, its experts on ``device``."""
    L = layer if isinstance(layer, Layer) else Layer.from_dict(layer)
    for name in ("gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s"):
        t = getattr(L, name)
        if t.device != device:
            raise FgmError(f"{name}: expected a tensor on {device}, got {t.device}")
    return L.struct()


def _token_rows(name: str, t: torch.Tensor, heads: int, D: int, device) -> int:
    """bf16 [B, N, heads, D] whose tokens are dense and evenly spaced over the
    whole batch (a slice of a fused projection's output qualifies); returns the
    elements between tokens."""
    if t.dtype is not _BF16 or t.dim() != 4 or t.shape[2] != heads or t.shape[3] != D or t.device != device:
        raise FgmError(f"{name}: expected bf16 [B, N, {heads}, {D}] on {device}, got {tuple(t.shape)} {t.dtype} "
                       f"on {t.device}")
    if t.is_contiguous():
        return heads * D
    B, N = t.shape[0], t.shape[1]
    sb, sn, sh, sd = t.stride()
    if (sd != 1) or (heads > 1 and sh != D):
        raise FgmError(f"{name}: a token's heads must be contiguous, strides {t.stride()}")
    if N > 1 and B > 1 and sb != N * sn:
        raise FgmError(f"{name}: sequences must follow each other at N token strides, strides {t.stride()}")
    return sn if N > 1 else sb if B > 1 else heads * D


def _table(B: int, block_table: torch.Tensor | None, C: fgm_kv_cache, device) -> tuple[int, int | None]:
    """(max_blocks, address) of a block table; without one each sequence owns an
    equal run of the cache's blocks."""
    if block_table is None:
        if C.n_blocks < B:
            raise FgmError(f"without a block_table the cache's {C.n_blocks} blocks are dealt to {B} sequences: too few")
        return C.n_blocks // B if B else 1, None
    if block_table.dim() != 2:
        raise FgmError(f"block_table: expected int32 [{B}, max_blocks], got {tuple(block_table.shape)}")
    mb = block_table.shape[1]
    return mb, _expect("block_table", block_table, (B, mb), _I32, device)


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, lens: torch.Tensor,
              block_table: torch.Tensor | None = None, ws: Workspace | None = None, stream=None) -> None:
    """Quantises the bf16 keys and values [B, N, kv heads, D] of each sequence's
    last N tokens into the cache. lens int32 [B]: tokens per sequence, the new
    ones included; block_table int32 [B, max_blocks] or None (each sequence owns
    an equal run of blocks)."""
    C, dev = cache.struct(), cache.v_q.device
    step = _token_rows("k", k, C.n_kv_heads, C.head_dim, dev)
    if _token_rows("v", v, C.n_kv_heads, C.head_dim, dev) != step or v.shape != k.shape:
        raise FgmError(f"k and v must have one shape and token stride, got {tuple(k.shape)} {k.stride()} and "
                       f"{tuple(v.shape)} {v.stride()}")
    B, N = k.shape[0], k.shape[1]
    mb, table = _table(B, block_table, C, dev)
    at = _expect("lens", lens, (B,), _I32, dev)

    def body(s):
        w = _space(ws, dev)
        _check(lib().fgm_kv_append(C, k.data_ptr(), v.data_ptr(), step, B, N, at, table, mb, w.t.data_ptr(), w.nbytes, s))
    _call(dev, stream, body)


def attn_workspace_bytes(B: int, M: int, n_q_heads: int, n_kv_heads: int, head_dim: int) -> int:
    """Workspace bytes of attn_fwd (0 when the sizes are not valid)."""
    return int(lib().fgm_attn_workspace_bytes(int(B), int(M), int(n_q_heads), int(n_kv_heads), int(head_dim)))


def attn_fwd(cache: KVCache, q: torch.Tensor, lens: torch.Tensor, scale: float,
             block_table: torch.Tensor | None = None, window: int = 0, out: torch.Tensor | None = None,
             lse: torch.Tensor | None = None, ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """Attention of bf16 q [B, M, q heads, D], the last M tokens of each sequence
    (already appended), over the cache; causal among them, with window > 0 over
    that many positions. Returns bf16 [B, M, q heads, D]; lse fp32 [B, M, q
    heads] receives the log of each row's sum of exponentials."""
    C, dev = cache.struct(), cache.v_q.device
    if window < 0:
        raise FgmError(f"window = {window}: 0 (none) or a positive number of tokens")
    window = min(window, 1 << 30)       # (no sequence is longer; a C int holds it)
    if q.dim() != 4:
        raise FgmError(f"q: expected bf16 [B, M, q heads, D], got {tuple(q.shape)}")
    B, M, Hq, D = q.shape
    step = _token_rows("q", q, Hq, C.head_dim, dev)
    mb, table = _table(B, block_table, C, dev)
    at = _expect("lens", lens, (B,), _I32, dev)
    lse_at = None if lse is None else _expect("lse", lse, (B, M, Hq), _F32, dev)

    def body(s):
        o = torch.empty((B, M, Hq, D), dtype=_BF16, device=dev) if out is None else out
        w = _space(ws, dev, attn_workspace_bytes, B, M, Hq, C.n_kv_heads, D)
        _check(lib().fgm_attn_fwd(C, q.data_ptr(), step, B, M, Hq, at, table, mb, scale, window,
                                  _expect("out", o, (B, M, Hq, D), _BF16, dev), lse_at, w.t.data_ptr(), w.nbytes, s))
        return o
    return _call(dev, stream, body)


# ---------------------------------------------------------------- log probabilities
class LogProbs(NamedTuple):
    """Per row: ln p of the given token, entropy (both fp32 [N]), and the k most
    likely words with their ln p (int32 and fp32 [N, k]); None where not asked for."""
    logp: torch.Tensor | None
    entropy: torch.Tensor | None
    top_ids: torch.Tensor | None
    top_logp: torch.Tensor | None


_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _score_outs(N: int, k: int, tokens, entropy: bool, out: LogProbs | None, dev) -> LogProbs:
    """The outputs of a log-probability call: ``out``'s tensors, checked, or new ones."""
    if not 0 <= k <= MAX_TOP:
        raise FgmError(f"k = {k} outside [0, {MAX_TOP}]")
    if out is None:
        return LogProbs(None if tokens is None else torch.empty(N, dtype=_F32, device=dev),
                        torch.empty(N, dtype=_F32, device=dev) if entropy else None,
                        torch.empty((N, k), dtype=_I32, device=dev) if k else None,
                        torch.empty((N, k), dtype=_F32, device=dev) if k else None)
    for name, t, shape, dt, want in (("logp", out.logp, (N,), _F32, tokens is not None), ("entropy", out.entropy, (N,), _F32, entropy),
                                     ("top_ids", out.top_ids, (N, k), _I32, k > 0), ("top_logp", out.top_logp, (N, k), _F32, k > 0)):
        if want != (t is not None):
            raise FgmError(f"out.{name}: {'missing' if want else 'given'}, though the call {'asks' if want else 'does not ask'} for it")
        if want:
            _expect("out." + name, t, shape, dt, dev)
    return out


def _at(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def logprobs_workspace_bytes(N: int, V: int, k: int) -> int:
    """Workspace bytes of logprobs (0 for sizes out of range)."""
    return int(lib().fgm_logprobs_workspace_bytes(int(N), int(V), int(k)))


def logprobs(z: torch.Tensor, tokens: torch.Tensor | None = None, k: int = 0, T: float = 1.0, entropy: bool = True,
             out: LogProbs | None = None, ws: Workspace | None = None, stream=None) -> LogProbs:
    """Log probabilities of rows of logits z [N, V] (fp32, bf16 or fp16; rows
    dense, any distance apart) under softmax(z / T): of the given tokens (int32
    [N]), with entropies and the k most likely words."""
    if z.dim() != 2 or z.dtype not in _DTYPES or not z.is_cuda:
        raise FgmError(f"z: expected CUDA fp32, bf16 or fp16 [N, V], got {tuple(z.shape)} {z.dtype} on {z.device}")
    N, V = z.shape
    stride, one = z.stride()
    if (V > 1 and one != 1) or (N > 1 and stride < V):
        raise FgmError(f"z: expected dense rows that do not overlap, strides {z.stride()}")
    dev = z.device
    at = None if tokens is None else _expect("tokens", tokens, (N,), _I32, dev)

    def body(s):
        r = _score_outs(N, k, tokens, entropy, out, dev)
        w = _space(ws, dev, logprobs_workspace_bytes, N, V, k)
        _check(lib().fgm_logprobs(z.data_ptr(), _DTYPES[z.dtype], stride if N > 1 else V, N, V, T, at, k, _at(r.logp),
                                  _at(r.entropy), _at(r.top_ids), _at(r.top_logp), w.t.data_ptr(), w.nbytes, s))
        return r
    return _call(dev, stream, body)


def lm_head_logprobs_workspace_bytes(N: int, V: int, k: int) -> int:
    """Workspace bytes of lm_head_logprobs (0 for sizes out of range)."""
    return int(lib().fgm_lm_head_logprobs_workspace_bytes(int(N), int(V), int(k)))


def lm_head_logprobs(emb: torch.Tensor, h: torch.Tensor, tokens: torch.Tensor | None = None, k: int = 0, T: float = 1.0,
                     entropy: bool = True, out: LogProbs | None = None, ws: Workspace | None = None,
                     stream=None) -> LogProbs:
    """logprobs of the tied lm_head's logits emb . h of the bf16 rows h [N, 2816]
    (any N: a decoded token, a verify step, a scored text), which are not stored."""
    if not emb.is_cuda or emb.dim() != 2:
        raise FgmError(f"emb: expected CUDA bf16 [V, {HIDDEN}], got {tuple(emb.shape)} on {emb.device}")
    dev, V = emb.device, emb.shape[0]
    e_at = _expect("emb", emb, (V, HIDDEN), _BF16, dev)
    if h.dim() != 2:
        raise FgmError(f"h: expected bf16 [N, {HIDDEN}], got {tuple(h.shape)}")
    N = h.shape[0]
    h_at = _expect("h", h, (N, HIDDEN), _BF16, dev)
    at = None if tokens is None else _expect("tokens", tokens, (N,), _I32, dev)

    def body(s):
        r = _score_outs(N, k, tokens, entropy, out, dev)
        w = _space(ws, dev, lm_head_logprobs_workspace_bytes, N, V, k)
        _check(lib().fgm_lm_head_logprobs(e_at, V, h_at, N, T, at, k, _at(r.logp), _at(r.entropy), _at(r.top_ids),
                                          _at(r.top_logp), w.t.data_ptr(), w.nbytes, s))
        return r
    return _call(dev, stream, body)


# ---------------------------------------------------------------- a prompt through the experts
class Routing(NamedTuple):
    """Of T tokens: chosen experts int32 [T, 8], their weights fp32 [T, 8], and the
    slots 8 * token + choice grouped by expert: offsets int32 [129], order int32 [8 T]."""
    ids: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor
    order: torch.Tensor


def _dense_rows(name: str, t: torch.Tensor, width: int | None, device=None) -> int:
    """Elements between the rows of a bf16 [n, width] tensor with dense rows."""
    if t.dtype is not _BF16 or t.dim() != 2 or (width is not None and t.shape[1] != width) or not t.is_cuda or \
            (device is not None and t.device != device):
        raise FgmError(f"{name}: expected CUDA bf16 [n, {'K' if width is None else width}]"
                       f"{'' if device is None else f' on {device}'}, got {tuple(t.shape)} {t.dtype} on {t.device}")
    n, w = t.shape
    sn, sw = t.stride()
    if w > 1 and sw != 1 or n > 1 and sn < w:
        raise FgmError(f"{name}: expected dense rows that do not overlap, strides {t.stride()}")
    return sn if n > 1 else (w + 7) // 8 * 8


def moe_route_workspace_bytes(T: int) -> int:
    """Workspace bytes of moe_route (0 for sizes out of range)."""
    return int(lib().fgm_moe_route_workspace_bytes(int(T)))


def moe_route(router_w: torch.Tensor, x: torch.Tensor, router_b: torch.Tensor | None = None, out: Routing | None = None,
              ws: Workspace | None = None, stream=None) -> Routing:
    """Routes the bf16 rows x [T, 2816] (any T): top 8 of 128 by the exact logits
    router_w . x + router_b, softmax over the 8, and the slots grouped by expert."""
    dev = x.device
    stride = _dense_rows("x", x, HIDDEN)
    T = x.shape[0]
    w_at = _expect("router_w", router_w, (EXPERTS, HIDDEN), _BF16, dev)
    b_at = None if router_b is None else _expect("router_b", router_b, (EXPERTS,), _F32, dev)

    if out is not None:
        for name, shape, dt in (("ids", (T, TOPK), _I32), ("weights", (T, TOPK), _F32), ("offsets", (EXPERTS + 1,), _I32),
                                ("order", (T * TOPK,), _I32)):
            _expect("out." + name, getattr(out, name), shape, dt, dev)

    def body(s):
        if out is None:
            r = Routing(torch.empty((T, TOPK), dtype=_I32, device=dev), torch.empty((T, TOPK), dtype=_F32, device=dev),
                        torch.empty(EXPERTS + 1, dtype=_I32, device=dev), torch.empty(T * TOPK, dtype=_I32, device=dev))
        else:
            r = out
        w = _space(ws, dev, moe_route_workspace_bytes, T)
        i, t, o, n = r
        _check(lib().fgm_moe_route(w_at, b_at, x.data_ptr(), stride, T, i.data_ptr(), t.data_ptr(), o.data_ptr(), n.data_ptr(),
                                   w.t.data_ptr(), w.nbytes, s))
        return r
    return _call(dev, stream, body)


def moe_group_workspace_bytes(n: int, E: int) -> int:
    """Workspace bytes of moe_group (0 for sizes out of range)."""
    return int(lib().fgm_moe_group_workspace_bytes(int(n), int(E)))


def moe_group(ids: torch.Tensor, E: int, offsets: torch.Tensor | None = None, order: torch.Tensor | None = None,
              ws: Workspace | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Groups the slots of int32 ids (any shape, flat order) by expert 0 .. E - 1: (offsets
    int32 [E + 1], order int32 [slots]); ids outside belong to none, and the places
    behind the last expert's are not written."""
    dev = ids.device
    if not ids.is_cuda:
        raise FgmError("expected a CUDA tensor")
    n = ids.numel()
    at = _expect("ids", ids, tuple(ids.shape), _I32, dev)

    def body(s):
        o = torch.empty(E + 1, dtype=_I32, device=dev) if offsets is None else offsets
        r = torch.empty(n, dtype=_I32, device=dev) if order is None else order
        w = _space(ws, dev, moe_group_workspace_bytes, n, E)
        _check(lib().fgm_moe_group(at, n, E, _expect("offsets", o, (E + 1,), _I32, dev), _expect("order", r, (n,), _I32, dev),
                                   w.t.data_ptr(), w.nbytes, s))
        return o, r
    if not 1 <= E <= MAX_GROUPS:
        raise FgmError(f"E = {E} outside [1, {MAX_GROUPS}]")
    return _call(dev, stream, body)


def grouped_gemm_workspace_bytes(x_rows: int, R: int, E: int, N: int, K: int) -> int:
    """Workspace bytes of grouped_gemm (0 for sizes out of range)."""
    return int(lib().fgm_grouped_gemm_workspace_bytes(int(x_rows), int(R), int(E), int(N), int(K)))


def grouped_gemm(x: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor | None, offsets: torch.Tensor,
                 rows: torch.Tensor | None = None, per: int = 1, out: torch.Tensor | None = None,
                 ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """Products grouped by expert: rows offsets[e] .. offsets[e + 1] of the result are
    bf16 x[rows // per] (or x itself) times w[e] [N, K] transposed, times w_s[e]. w is uint8
    [E, N, K] E4M3 codes or bf16; w_s fp32 [E, N] or None. Returns bf16 [R, N], whose rows of
    no expert are as they were in ``out``."""
    dev = x.device
    stride = _dense_rows("x", x, None)
    if w.dim() != 3 or w.dtype not in (_U8, _BF16):
        raise FgmError(f"w: expected uint8 (E4M3) or bf16 [E, N, K], got {tuple(w.shape)} {w.dtype}")
    E, N, K = w.shape
    if x.shape[1] != K:
        raise FgmError(f"x: expected rows of K = {K}, got {tuple(x.shape)}")
    w_at = _expect("w", w, (E, N, K), w.dtype, dev)
    s_at = None if w_s is None else _expect("w_s", w_s, (E, N), _F32, dev)
    o_at = _expect("offsets", offsets, (E + 1,), _I32, dev)
    if rows is not None and rows.dim() != 1:
        raise FgmError(f"rows: expected int32 [R], got {tuple(rows.shape)}")
    R = x.shape[0] if rows is None else rows.shape[0]
    r_at = None if rows is None else _expect("rows", rows, (R,), _I32, dev)

    if out is not None:
        _expect("out", out, (R, N), _BF16, dev)

    def body(s):
        o = torch.empty((R, N), dtype=_BF16, device=dev) if out is None else out
        v = _space(ws, dev, grouped_gemm_workspace_bytes, x.shape[0], R, E, N, K) if w.dtype is _U8 else _space(ws, dev)
        _check(lib().fgm_grouped_gemm(x.data_ptr(), stride, x.shape[0], r_at, per, o_at, w_at, E4M3 if w.dtype is _U8 else 1, s_at,
                                      E, N, K, o.data_ptr(), R, v.t.data_ptr(), v.nbytes, s))
        return o
    return _call(dev, stream, body)


def moe_experts_workspace_bytes(T: int) -> int:
    """Workspace bytes of moe_experts_fwd (0 for sizes out of range)."""
    return int(lib().fgm_moe_experts_workspace_bytes(int(T)))


def moe_experts_fwd(layer, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, y: torch.Tensor | None = None,
                    shared: bool = True, ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """A layer's experts on the bf16 rows x [T, 2816] (any T), each token's experts
    int32 ids [T, 8] (outside [0, 128): none) weighted by fp32 weights [T, 8], plus
    the shared expert; returns bf16 y [T, 2816]."""
    dev = x.device
    stride = _dense_rows("x", x, HIDDEN)
    T = x.shape[0]
    L = _layer_on(layer, dev)
    i_at = _expect("ids", ids, (T, TOPK), _I32, dev)
    w_at = _expect("weights", weights, (T, TOPK), _F32, dev)

    def body(s):
        o = torch.empty((T, HIDDEN), dtype=_BF16, device=dev) if y is None else y
        w = _space(ws, dev, moe_experts_workspace_bytes, T)
        _check(lib().fgm_moe_experts_fwd(ctypes.byref(L), x.data_ptr(), stride, T, i_at, w_at, int(shared),
                                         _expect("y", o, (T, HIDDEN), _BF16, dev), w.t.data_ptr(), w.nbytes, s))
        return o
    return _call(dev, stream, body)


def _norm_rows(name: str, t: torch.Tensor, shape, device) -> tuple[int, int, int]:
    """(address, type, elements between rows) of a tensor with dense rows."""
    kind = _DTYPES.get(t.dtype)
    if kind is None or t.shape != shape or t.device != device:
        raise FgmError(f"{name}: expected fp32, bf16 or fp16 {tuple(shape)} on {device}, got {tuple(t.shape)} {t.dtype} on {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), kind, shape[1]
    sn, sd = t.stride()
    if shape[1] > 1 and sd != 1:
        raise FgmError(f"{name}: expected dense rows, strides {t.stride()}")
    return t.data_ptr(), kind, sn if shape[0] > 1 else max(sn, shape[1])


def _gain(t: torch.Tensor, D: int, device, dtype) -> tuple[int, int]:
    """(address, type) of a norm's gains."""
    kind = _DTYPES.get(t.dtype)
    if kind is None or t.shape != (D,) or t.device != device or not t.is_contiguous() or t.dtype is not dtype:
        raise FgmError(f"gains: expected contiguous [{D}] of one type on {device}, got {tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr(), kind


def block_norm(h: torch.Tensor, y: torch.Tensor | None = None, post_gain: torch.Tensor | None = None,
               gate: torch.Tensor | None = None, pre_gain: torch.Tensor | None = None, post_norm: bool = True,
               pre_norm: bool = True, residual_scale: float = 1.0, block_scale: float = 1.0, gain_offset: float = 0.0,
               eps: float = 1e-6, h_out: torch.Tensor | None = None, xn: torch.Tensor | None = None,
               stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """The norms around a block: h' = residual_scale * h + block_scale * gate * post(y) and
    xn = pre(h') (RMS norms with gains post_gain, pre_gain [D]); gate [D] a channel, [N, 1] a
    token or [N, D]. Returns (h', xn): h' in h's type (``h_out`` may be h), xn in bf16 or in the type of
    ``xn``; xn is None without pre_norm."""
    if h.dim() != 2 or not h.is_cuda:
        raise FgmError(f"h: expected CUDA [N, D], got {tuple(h.shape)} on {h.device}")
    dev, shape = h.device, h.shape
    N, D = shape
    h_at, h_type, h_step = _norm_rows("h", h, shape, dev)
    y_at, y_type, y_step = (None, 0, 0) if y is None else _norm_rows("y", y, shape, dev)
    g_at = g_type = g_rows = g_cols = 0
    if gate is not None:
        if gate.dtype not in _DTYPES or gate.device != dev or tuple(gate.shape) not in ((D,), (N, 1), (N, D)):
            raise FgmError(f"gate: expected [{D}], [{N}, 1] or [{N}, {D}] on {dev}, got {tuple(gate.shape)} {gate.dtype} on {gate.device}")
        g_cols = int(gate.dim() == 1 or gate.shape[1] != 1 or D == 1)
        if g_cols and D > 1 and gate.stride(-1) != 1:
            raise FgmError(f"gate: expected dense rows, strides {gate.stride()}")
        g_at, g_type = gate.data_ptr(), _DTYPES[gate.dtype]
        g_rows = gate.stride(0) if gate.dim() == 2 and N > 1 else 0
    gain_type, p_at, q_at = 0, None, None
    if post_gain is not None:
        p_at, gain_type = _gain(post_gain, D, dev, post_gain.dtype)
    if pre_gain is not None:
        q_at, gain_type = _gain(pre_gain, D, dev, pre_gain.dtype if post_gain is None else post_gain.dtype)
    if xn is not None and not pre_norm:
        raise FgmError("xn without pre_norm")

    def body(s):
        if h_out is None:
            o = torch.empty(shape, dtype=h.dtype, device=dev)
            o_at, o_step = o.data_ptr(), D
        else:
            o = h_out
            o_at, o_type, o_step = _norm_rows("h_out", o, shape, dev)
            if o_type != h_type:
                raise FgmError(f"h_out: expected {h.dtype}, got {o.dtype}")
        n, n_at, n_type, n_step = xn, None, 0, 0
        if xn is not None:
            n_at, n_type, n_step = _norm_rows("xn", n, shape, dev)
        elif pre_norm:
            n = torch.empty(shape, dtype=_BF16, device=dev)
            n_at, n_type, n_step = n.data_ptr(), 1, D
        _check(lib().fgm_block_norm(fgm_block(
            N, D, h_type, y_type, g_type, gain_type, n_type, h_at, y_at, g_at, p_at, q_at, o_at, n_at, h_step,
            y_step, g_rows, o_step, n_step, g_cols, post_norm and y is not None, residual_scale, block_scale, gain_offset, eps), s))
        return o, n
    return _call(dev, stream, body)
