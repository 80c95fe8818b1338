"""Plain 64-bit forms of the routing, grouped products, experts and block norms, on
torch tensors, with bounds of the errors that the operators' documented precision allows."""

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}     # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # of values near zero
ADD = 2.0 ** -22                 # an addition of the tensor pipe, of the sum of what it has added
TERM = 2.0 ** -17                # two E4M3 terms of a bf16 element, of its row's largest


def e4m3(q):
    return q.view(torch.float8_e4m3fn).double()


def group(ids, E):
    """offsets and order of flat ids, others than 0 .. E - 1 left out."""
    ids = ids.reshape(-1).tolist()
    order = [[] for _ in range(E)]
    for i, e in enumerate(ids):
        if 0 <= e < E:
            order[e].append(i)
    offsets = [0]
    for o in order:
        offsets.append(offsets[-1] + len(o))
    return offsets, [i for o in order for i in o]


def route(w, x, b, k=8):
    """ids and weights by exact logits (fp64: 2^-40 of a sum is far below what the tests tell apart), and |x| |w|."""
    z = x.double() @ w.double().t()
    if b is not None:
        z = z + b.double()
    z = torch.where(torch.isnan(z), -math.inf, z)
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    top = z.gather(1, ids)
    return ids, torch.softmax(top, dim=1), top


def products(x, w, s, e4m3_x):
    """rows of x [R, K] times w [N, K] (fp64 values) transposed, times s [N]: the result and a bound of the accumulator's error."""
    x64 = x.double()
    d, a = x64 @ w.t(), x64.abs() @ w.abs().t()
    K = x.shape[1]
    adds = 2 * ((K + 31) // 32) if e4m3_x else (K + 15) // 16
    err = adds * ADD * a
    if e4m3_x:
        err = err + TERM * x64.abs().amax(dim=1, keepdim=True) * w.abs().sum(dim=1)
    return d * s, err * s.abs()


def rounded(v, err, dtype):
    """Bound of v + err rounded to a type."""
    return err + (v.abs() + err) * HALF[dtype] * 1.01 + TINY[dtype]


def gelu(g):
    return torch.nn.functional.gelu(g, approximate="tanh")


def experts(L, x, ids, weights, shared):
    """y and a bound of its error before the last rounding; L: fp64 copies not needed, codes and scales as given."""
    x64, T = x.double(), x.shape[0]
    y, bound = torch.zeros_like(x64), torch.zeros_like(x64)
    jobs = [(e, (ids == e).nonzero()) for e in range(128)] + ([(128, None)] if shared else [])
    for e, at in jobs:
        t = torch.arange(T, device=x.device) if at is None else at[:, 0]
        if len(t) == 0:
            continue
        wt = torch.ones(len(t), dtype=torch.float64, device=x.device) if at is None else weights[at[:, 0], at[:, 1]].double()
        g, dg = products(x[t], e4m3(L["gate_q"][e]), L["gate_s"][e].double(), True)
        u, du = products(x[t], e4m3(L["up_q"][e]), L["up_s"][e].double(), True)
        a = gelu(g) * u
        # gelu' is at most 1.13; its own evaluation 2^-20; f16 and the two terms 2^-9 and 2^-11 of a, or of the row's largest 2^-17
        da = 1.13 * dg * (u.abs() + du) + gelu(g).abs() * du + (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -20) * a.abs() + TERM * a.abs().amax(dim=1, keepdim=True)
        w, s = e4m3(L["down_q"][e]), L["down_s"][e].double()
        o = (a @ w.t()) * s
        do = (da @ w.abs().t() + 44 * ADD * (a.abs() @ w.abs().t())) * s.abs()
        do = do + 2.0 ** -11 * (o.abs() + do) + 2.0 ** -36 * s.abs().max() * a.abs().amax(dim=1, keepdim=True) * 448 * 704
        y.index_add_(0, t, o * wt[:, None])
        bound.index_add_(0, t, do * wt.abs()[:, None] + 2.0 ** -21 * (o * wt[:, None]).abs())
    return y, bound


def block(h, y, post, gate, pre, post_norm, a, b, offset, eps):
    """h' and xn in 64 bits; bounds of what fp32 sums and products may be off (2^-18 of the parts)."""
    h64 = h.double()
    part = torch.zeros_like(h64)
    if y is not None:
        part = y.double()
        if post_norm:
            part = part / torch.sqrt(part.square().mean(dim=1, keepdim=True) + eps)
        if post is not None:
            part = part * (post.double() + offset)
        if gate is not None:
            part = part * gate.double()
    out = a * h64 + b * part
    dout = 2.0 ** -18 * ((a * h64).abs() + (b * part).abs())
    r = 1.0 / torch.sqrt(out.square().mean(dim=1, keepdim=True) + eps)
    g = torch.ones_like(out) if pre is None else (pre.double() + offset).expand_as(out)
    xn = out * r * g
    # the sum of squares is off by 2^-18 of itself and by what h' is; half of that in the root
    dr = r * (2.0 ** -18 + (out * dout).abs().sum(dim=1, keepdim=True) / out.square().sum(dim=1, keepdim=True).clamp_min(1e-300))
    return out, dout, xn, (dout * r + out.abs() * dr) * g.abs() + 2.0 ** -20 * xn.abs()


def within(got, want, bound):
    """Whether got is within the bound of want; NaN only where want is."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = torch.isnan(want) | ((got - want).abs() <= bound) | (got == want)
    assert ok.all(), (float((got - want).abs()[~ok].max()), int((~ok).sum()), (~ok).nonzero()[:5].tolist())
