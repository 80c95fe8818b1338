"""The measured cases of a prompt's way through a layer's experts: routing, products
grouped by expert, the experts' weighted sum, and the norms around a block.

``run`` makes one pass through an operator: in plain torch operations where
``own`` is false, through the package's entry points where it is true.
``exact`` restates each operator in 64 bits.

Tensors. Expert weights are E4M3 codes in uint8 with an fp32 scale per output
row (or bf16 without scales); activations are bf16. A slot is a (token, choice)
pair, numbered 8 * token + choice; ``order`` lists slots by expert, and
``offsets[e] .. offsets[e + 1]`` are expert e's places in it.
"""

from __future__ import annotations

import math

import torch

own = False

HIDDEN = 2816       # hidden width of the model
FFN = 704           # width of an expert
EXPERTS = 128       # routed experts (a shared one is stored behind them)
TOPK = 8
EPS = 1e-6


def listed():
    return [
        # the 5 tokens of one verify step: chosen experts, weights and their grouping
        dict(name="route_verify", op="route", T=5, zipf=1.1),
        # a long prompt
        dict(name="route_prompt", op="route", T=16381, zipf=1.1),
        # gate products of a few requests' tokens: 8 slots a token, gathered from the tokens' rows
        dict(name="gemm_requests", op="gemm", E=128, N=704, K=2816, T=26, per=8, zipf=1.1, weights="e4m3"),
        # down products of a prompt's slots, rows in order of the experts
        dict(name="gemm_prompt", op="gemm", E=128, N=2816, K=704, T=32771, per=0, zipf=1.1, weights="e4m3"),
        # fewer and wider experts in bf16 (an adapter's, or a draft model's)
        dict(name="gemm_bf16", op="gemm", E=16, N=2112, K=1408, T=4507, per=2, zipf=0.5, weights="bf16"),
        # a decoded token through a layer's experts
        dict(name="experts_token", op="experts", T=1, zipf=1.1, pad=0),
        # a batch of requests, a token each, some places of it empty
        dict(name="experts_batch", op="experts", T=61, zipf=1.1, pad=7),
        # a chat turn
        dict(name="experts_turn", op="experts", T=1021, zipf=1.1, pad=0),
        # a long prompt
        dict(name="experts_prompt", op="experts", T=16381, zipf=1.1, pad=0),
        # the residual stream of a verify step: the block's norm, the sum, the next block's norm
        dict(name="norm_verify", op="norm", N=5, D=2816, h="float32", y="bfloat16", gate="none", post=True, pre=True, scale=1.0),
        # the same of a long prompt, with the layer's scale
        dict(name="norm_prompt", op="norm", N=16381, D=2816, h="bfloat16", y="bfloat16", gate="none", post=True, pre=True,
             scale=0.73),
        # a gate per element, rows of an odd width
        dict(name="norm_gated", op="norm", N=4099, D=1409, h="float32", y="bfloat16", gate="full", post=True, pre=True, scale=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "gemm", "gemm", "experts", "experts", "norm"])
    zipf = rng.choice([0.0, 0.5, 1.1, 2.0])
    if op == "route":
        return dict(op=op, T=_log_int(rng, 1, 16000), zipf=zipf)
    if op == "gemm":
        weights = rng.choice(["e4m3", "e4m3", "bf16"])
        E = rng.choice([1, 8, 16, 60, 128])
        K = 16 * _log_int(rng, 2, 176)
        N = _log_int(rng, 8, 2816)
        T = _log_int(rng, 1, max(2, min(30000, int(6e10 / (K * N)))))
        return dict(op=op, E=E, N=N, K=K, T=T, per=rng.choice([0, 1, 2, 8]), zipf=zipf, weights=weights)
    if op == "experts":
        T = _log_int(rng, 1, 12000)
        return dict(op=op, T=T, zipf=zipf, pad=rng.choice([0, 0, T // 5]))
    D = rng.choice([HIDDEN, _log_int(rng, 33, 8192)])
    return dict(op=op, N=_log_int(rng, 1, max(2, 45_000_000 // D)), D=D, h=rng.choice(["float32", "bfloat16"]),
                y=rng.choice(["bfloat16", "float32", "float16"]), gate=rng.choice(["none", "channel", "token", "full"]),
                post=rng.random() < 0.8, pre=rng.random() < 0.8, scale=rng.choice([1.0, 0.73]))


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _hidden(T, g, width=HIDDEN):
    """Rows as a norm leaves them, a few channels strong."""
    x = torch.randn(T, width, generator=g, device="cuda")
    x[:, 5::331] *= 9.0
    return (x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)).bfloat16()


def _codes(E, rows, K, g):
    """E4M3 codes and row scales of weights ~N(0, 1 / 50), rows of uneven size."""
    q = torch.empty(E, rows, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, rows, device="cuda")
    step = max(1, (1 << 27) // (rows * K))
    for i in range(0, E, step):
        n = min(step, E - i)
        w = torch.randn(n, rows, K, generator=g, device="cuda") * 0.02
        w *= 0.5 + torch.rand(n, rows, 1, generator=g, device="cuda")
        s[i:i + n] = w.abs().amax(dim=2) / 448.0
        q[i:i + n] = (w / s[i:i + n, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q, s


def _choices(T, E, k, zipf, g):
    """k distinct experts of E a token, frequent ones first in the numbering, and their weights."""
    score = torch.randn(T, E, generator=g, device="cuda") - zipf * torch.log(torch.arange(E, device="cuda") + 1.0)
    top, ids = torch.topk(score, k, dim=1)
    return ids.to(torch.int32), torch.softmax(top, dim=1)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op == "route":
        st["x"] = _hidden(case["T"], g)
        st["router_w"] = (torch.randn(EXPERTS, HIDDEN, generator=g, device="cuda") * 0.02).bfloat16()
        st["router_b"] = -case["zipf"] * torch.log(torch.arange(EXPERTS, device="cuda") + 1.0)
    elif op == "gemm":
        T, E, N, K, per = case["T"], case["E"], case["N"], case["K"], case["per"]
        st["x"] = _hidden(T, g, K)
        if case["weights"] == "e4m3":
            st["w"], st["s"] = _codes(E, N, K, g)
        else:
            st["w"], st["s"] = (torch.randn(E, N, K, generator=g, device="cuda") * 0.02).bfloat16(), None
        if per:
            ids = _choices(T, E, min(per, E), case["zipf"], g)[0]
            ids = torch.cat([ids, ids[:, :1].expand(T, per - ids.shape[1])], dim=1).reshape(-1).long()
            order = torch.argsort(ids, stable=True)
            st["rows"], st["per"] = order.to(torch.int32), per
        else:
            ids = _choices(T, E, 1, case["zipf"], g)[0].reshape(-1).long()
            st["rows"], st["per"] = None, 1
        st["offsets"] = torch.nn.functional.pad(torch.cumsum(torch.bincount(ids, minlength=E), 0), (1, 0)).to(torch.int32)
    elif op == "experts":
        T = case["T"]
        st["x"] = _hidden(T, g)
        st["ids"], st["weights"] = _choices(T, EXPERTS, TOPK, case["zipf"], g)
        if case["pad"]:                          # places of a padded batch choose no expert
            st["ids"][torch.randperm(T, generator=g, device="cuda")[:case["pad"]]] = -1
        layer = {"router_w": torch.zeros(EXPERTS, HIDDEN, dtype=torch.bfloat16, device="cuda"), "router_b": None}
        for name, rows, K in (("gate", FFN, HIDDEN), ("up", FFN, HIDDEN), ("down", HIDDEN, FFN)):
            layer[name + "_q"], layer[name + "_s"] = _codes(EXPERTS + 1, rows, K, g)
        st["layer"] = layer
    else:
        N, D = case["N"], case["D"]
        st["y"] = (torch.randn(N, D, generator=g, device="cuda") * 0.3).to(getattr(torch, case["y"]))
        h = torch.randn(N, D, generator=g, device="cuda") * 2.0
        h[:, 3::257] *= 20.0
        st["h"] = h.to(getattr(torch, case["h"]))
        st["post"] = torch.rand(D, generator=g, device="cuda") + 0.5 if case["post"] else None
        st["pre"] = torch.rand(D, generator=g, device="cuda") + 0.5 if case["pre"] else None
        shape = {"none": None, "channel": (D,), "token": (N, 1), "full": (N, D)}[case["gate"]]
        st["gate"] = None if shape is None else torch.rand(shape, generator=g, device="cuda").bfloat16()
    if own:
        import fine_grained_moe_gb300 as fgm
        if op == "route":
            st["ws"] = fgm.Workspace("cuda", nbytes=fgm.moe_route_workspace_bytes(case["T"]))
        elif op == "gemm":
            R = T * max(1, per)
            st["ws"] = fgm.Workspace("cuda", nbytes=fgm.grouped_gemm_workspace_bytes(T, R, E, N, K))
        elif op == "experts":
            st["layer"] = fgm.Layer.from_dict(st["layer"])
            st["ws"] = fgm.Workspace("cuda", nbytes=fgm.moe_experts_workspace_bytes(T))
    return st


# ---------------------------------------------------------------- plain forms
def _top(z, k):
    """The k largest of each row of fp64 logits, ties to the lower index."""
    return torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]


def _route_plain(st):
    # (64 bits: whole numbers hang on logits that lie next to each other)
    z = torch.matmul(st["x"].double(), st["router_w"].double().t()) + st["router_b"].double()
    ids = _top(z, TOPK)
    top = z.gather(1, ids).float()
    e = torch.exp(top - top[:, :1])
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    count = torch.zeros(EXPERTS + 1, dtype=torch.int64, device=flat.device)
    count[1:].index_add_(0, flat, torch.ones_like(flat))
    return [ids.to(torch.int32), e / e.sum(dim=1, keepdim=True), torch.cumsum(count, 0).to(torch.int32), order.to(torch.int32)]


def _decoded(q, s):
    """fp32 weights of one expert."""
    return q.float() if s is None else q.view(torch.float8_e4m3fn).float() * s[:, None]


def _gemm_plain(st):
    x = st["x"] if st["rows"] is None else st["x"][(st["rows"] // st["per"]).long()]
    out = torch.empty(x.shape[0], st["w"].shape[1], dtype=torch.bfloat16, device=x.device)
    at = st["offsets"].tolist()
    for e in range(len(at) - 1):
        if at[e + 1] > at[e]:
            w = _decoded(st["w"][e], None if st["s"] is None else st["s"][e])
            out[at[e]:at[e + 1]] = torch.matmul(x[at[e]:at[e + 1]].float(), w.t()).bfloat16()
    return [out]


def _gelu(g):
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _expert_plain(L, e, x):
    a = _gelu(torch.matmul(x, _decoded(L["gate_q"][e], L["gate_s"][e]).t()))
    a = a * torch.matmul(x, _decoded(L["up_q"][e], L["up_s"][e]).t())
    return torch.matmul(a, _decoded(L["down_q"][e], L["down_s"][e]).t())


def _experts_plain(st):
    L, x = st["layer"], st["x"].float()
    flat = st["ids"].reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    count = torch.bincount(flat + 1, minlength=EXPERTS + 1).tolist()
    y = _expert_plain(L, EXPERTS, x)
    at = count[0]                                # (slots that name no expert come first)
    for e in range(EXPERTS):
        slots = order[at:at + count[e + 1]]
        at += count[e + 1]
        if count[e + 1]:
            t = slots // TOPK
            y.index_add_(0, t, _expert_plain(L, e, x[t]) * st["weights"].reshape(-1)[slots][:, None])
    return [y.bfloat16()]


def _norm_plain(st):
    c = st["case"]
    y, h = st["y"].float(), st["h"].float()
    if c["post"]:
        y = y * torch.rsqrt((y * y).mean(dim=1, keepdim=True) + EPS) * st["post"]
    if st["gate"] is not None:
        y = y * st["gate"].float()
    h = c["scale"] * (h + y)
    out = [h.to(st["h"].dtype)]
    if c["pre"]:
        out.append((h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * st["pre"]).bfloat16())
    return out


def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        return {"route": _route_plain, "gemm": _gemm_plain, "experts": _experts_plain, "norm": _norm_plain}[op](st)
    import fine_grained_moe_gb300 as fgm
    if op == "route":
        return list(fgm.moe_route(st["router_w"], st["x"], st["router_b"], ws=st["ws"]))
    if op == "gemm":
        return [fgm.grouped_gemm(st["x"], st["w"], st["s"], st["offsets"], rows=st["rows"], per=st["per"], ws=st["ws"])]
    if op == "experts":
        return [fgm.moe_experts_fwd(st["layer"], st["x"], st["ids"], st["weights"], ws=st["ws"])]
    h, xn = fgm.block_norm(st["h"], st["y"], post_gain=st["post"], post_norm=c["post"], gate=st["gate"], pre_gain=st["pre"],
                           pre_norm=c["pre"], residual_scale=c["scale"], block_scale=c["scale"], eps=EPS)
    return [h, xn] if c["pre"] else [h]


# ---------------------------------------------------------------- work
def _active(T, E, k, zipf):
    """Experts that T tokens are expected to reach, each choosing k of E by the shares of a Zipf law."""
    p = [(e + 1.0) ** -zipf for e in range(E)]
    share = [min(1.0, k * v / sum(p)) for v in p]
    return max(min(k, E), sum(1.0 - (1.0 - v) ** T for v in share))


def work(case):
    op = case["op"]
    if op == "route":
        T = case["T"]
        return {"bytes": 2 * HIDDEN * (T + EXPERTS) + T * TOPK * 12 + 8 * EXPERTS, "flops": 2 * HIDDEN * EXPERTS * T}
    if op == "gemm":
        T, E, N, K, per = case["T"], case["E"], case["N"], case["K"], case["per"]
        R = T * max(1, per)
        one = N * K + 4 * N if case["weights"] == "e4m3" else 2 * N * K
        return {"bytes": _active(T, E, max(1, per), case["zipf"]) * one + 2 * T * K + 2 * R * N + (4 * R if per else 0),
                "flops": 2 * R * N * K}
    if op == "experts":
        T, live = case["T"], case["T"] - case["pad"]
        one = 3 * FFN * HIDDEN + 4 * (2 * FFN + HIDDEN)
        return {"bytes": (_active(live, EXPERTS, TOPK, case["zipf"]) + 1) * one + T * (4 * HIDDEN + 8 * TOPK),
                "flops": 2 * 3 * FFN * HIDDEN * (TOPK * live + T)}
    N, D = case["N"], case["D"]
    size = {"float32": 4, "bfloat16": 2, "float16": 2}
    gate = {"none": 0, "channel": D, "token": N, "full": N * D}[case["gate"]]
    return {"bytes": N * D * (size[case["y"]] + 2 * size[case["h"]] + 2 * case["pre"]) + 2 * gate
            + 4 * D * (case["post"] + case["pre"]), "flops": 10 * N * D}


# ---------------------------------------------------------------- 64 bits
def _exact_route(st):
    z = torch.einsum("th,eh->te", st["x"].double(), st["router_w"].double()) + st["router_b"].double()
    rank = torch.argsort(-z, dim=1, stable=True)[:, :TOPK]
    w = torch.softmax(torch.take_along_dim(z, rank, 1), dim=1)
    slots = [[] for _ in range(EXPERTS)]
    for i, e in enumerate(rank.reshape(-1).tolist()):
        slots[e].append(i)
    at = [0]
    for s in slots:
        at.append(at[-1] + len(s))
    return [rank.int(), w, torch.tensor(at, dtype=torch.int32), torch.tensor(sum(slots, []), dtype=torch.int32)]


def _dequant(q, s):
    return q.double() if s is None else torch.einsum("n,nk->nk", s.double(), q.view(torch.float8_e4m3fn).double())


def _exact_gemm(st):
    at = st["offsets"].tolist()
    parts = []
    for e in range(st["w"].shape[0]):
        r = torch.arange(at[e], at[e + 1], device="cuda")
        if st["rows"] is not None:
            r = torch.div(st["rows"].long()[r], st["per"], rounding_mode="floor")
        w = _dequant(st["w"][e], None if st["s"] is None else st["s"][e]) if len(r) else st["w"][e].double()
        parts.append(st["x"][r].double() @ w.t())
    return [torch.cat(parts)]


def _exact_experts(st):
    L, x = st["layer"], st["x"].double()
    y = torch.zeros_like(x)
    gate = torch.zeros(x.shape[0], EXPERTS + 1, dtype=torch.float64, device="cuda")
    ids = st["ids"].long()
    gate.scatter_add_(1, torch.where(ids < 0, EXPERTS, ids), torch.where(ids < 0, torch.zeros_like(st["weights"]), st["weights"]).double())
    chosen = torch.zeros_like(gate, dtype=torch.bool).scatter_(1, torch.where(ids < 0, EXPERTS, ids), True)
    gate[:, EXPERTS], chosen[:, EXPERTS] = 1.0, True
    for e in range(EXPERTS + 1):
        t = chosen[:, e].nonzero()[:, 0]
        if len(t) == 0:
            continue
        gate_w, up_w, down_w = (_dequant(L[n + "_q"][e], L[n + "_s"][e]) for n in ("gate", "up", "down"))
        a = torch.nn.functional.gelu(x[t] @ gate_w.t(), approximate="tanh") * (x[t] @ up_w.t())
        y[t] += gate[t, e][:, None] * (a @ down_w.t())
    return [y]


def _exact_norm(st):
    c = st["case"]
    y, h = st["y"].double(), st["h"].double()
    if c["post"]:
        y = y / torch.sqrt(y.square().mean(dim=1, keepdim=True) + EPS) * st["post"].double()
    if st["gate"] is not None:
        y = y * st["gate"].double()
    h = c["scale"] * h + c["scale"] * y
    return [h] + ([h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + EPS) * st["pre"].double()] if c["pre"] else [])


def exact(case, seed):
    st = prepare(case, seed)
    if own and case["op"] == "experts":
        st["layer"] = vars(st["layer"])
    return {"route": _exact_route, "gemm": _exact_gemm, "experts": _exact_experts, "norm": _exact_norm}[case["op"]](st)
