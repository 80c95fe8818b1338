"""The measured cases of the 8-bit KV cache, its attention and the log probabilities.

``run`` makes one pass through an operator: in plain torch operations where
``own`` is false, through the package's entry points where it is true.
``exact`` restates each operator in 64 bits.

Tensors. A cache holds blocks of 64 tokens: K codes [blocks, kv heads, D / 64,
64 tokens, 64 dims], V codes [blocks, kv heads, D, 64 tokens], both E4M3 in
uint8, and one fp32 scale per block and kv head for each. ``lens`` counts a
sequence's tokens including those of the call.
"""

from __future__ import annotations

import math

import torch

own = False

BLOCK = 64          # tokens per cache block
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -60
HIDDEN = 2816       # hidden width of the model
VOCAB = 262144      # its vocabulary


def listed():
    return [
        # K/V of the 5 tokens of one verify step (4 drafts), one layer, behind a 4,093-token context
        dict(name="append_verify", op="append", B=1, N=5, H=8, D=256, lens="4098"),
        # K/V of a long prompt written into a fresh cache at once
        dict(name="append_prompt", op="append", B=1, N=16381, H=8, D=256, lens="16381"),
        # plain decoding (one token) of a chat turn of 1,000 tokens
        dict(name="attn_decode_short", op="attn", B=1, M=1, H=8, G=2, D=256, lens="1000", window=0),
        # a sliding-window layer of the verify step deep into a context
        dict(name="attn_verify_window", op="attn", B=1, M=5, H=8, G=2, D=256, lens="40007", window=1024),
        # a full-attention layer of the verify step at 32K tokens
        dict(name="attn_verify_32k", op="attn", B=1, M=5, H=8, G=2, D=256, lens="32771", window=0),
        # the same at the longest context, few kv heads: 40 query rows share a head's cache
        dict(name="attn_verify_256k", op="attn", B=1, M=5, H=2, G=8, D=256, lens="262139", window=0),
        # one token each for requests of uneven lengths
        dict(name="attn_decode_ragged", op="attn", B=9, M=1, H=8, G=4, D=128,
             lens="16001 1 777 12345 64 8191 30011 4097 129", window=0),
        # the logits of one verify step: log probability of each emitted token, entropy, 8 alternatives
        dict(name="logprobs_verify", op="logprobs", N=5, V=VOCAB, k=8, T=1.0, dtype="float32"),
        # stored bf16 logits of a batch with an odd vocabulary, at a temperature
        dict(name="logprobs_batch", op="logprobs", N=1013, V=50021, k=5, T=0.7, dtype="bfloat16"),
        # logits of a scored passage
        dict(name="logprobs_passage", op="logprobs", N=600, V=VOCAB, k=1, T=1.0, dtype="float32"),
        # one verify step from its hidden rows
        dict(name="lm_head_verify", op="lm_head", N=5, V=VOCAB, k=8, T=1.0),
        # a scored prompt from its hidden rows
        dict(name="lm_head_prompt", op="lm_head", N=1021, V=VOCAB, k=4, T=1.0),
    ]


def _lens(case):
    return [int(n) for n in case["lens"].split()]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "logprobs", "lm_head"])
    if op == "append":
        B, H, D = rng.randint(1, 6), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        N = rng.randint(1, 8) if rng.random() < 0.5 else _log_int(rng, 9, 4000)
        return dict(op=op, B=B, N=N, H=H, D=D, lens=" ".join(str(N + rng.randint(0, 3000)) for _ in range(B)))
    if op == "attn":
        D, H = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8])
        M = rng.randint(1, 8)
        G = rng.choice([g for g in (1, 2, 4, 6, 8, 16) if g * M <= 64])
        B = rng.randint(1, 12)
        top = min(262144, 16_000_000 // (B * H) * 16 // D)
        lens = " ".join(str(_log_int(rng, M, max(M + 1, top))) for _ in range(B))
        return dict(op=op, B=B, M=M, H=H, G=G, D=D, lens=lens, window=rng.choice([0, 0, 1024, rng.randint(1, 5000)]))
    if op == "logprobs":
        V = rng.choice([VOCAB, _log_int(rng, 500, 262143)])
        return dict(op=op, N=_log_int(rng, 1, max(2, 140_000_000 // V)), V=V, k=rng.randint(0, 16),
                    T=rng.choice([1.0, 0.7, 1.3]), dtype=rng.choice(["float32", "bfloat16", "float16"]))
    V = rng.choice([VOCAB, _log_int(rng, 4000, 262143)])
    return dict(op=op, N=_log_int(rng, 1, 1000), V=V, k=rng.randint(0, 4), T=rng.choice([1.0, 0.8]))


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _table(case, g):
    """Block table of shuffled physical blocks, as a pool hands them out after a while, and the pool's size."""
    per = max((n + BLOCK - 1) // BLOCK for n in _lens(case))
    total = case["B"] * per + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    return perm[:case["B"] * per].view(case["B"], per).contiguous(), total


def _quantised(x):
    """[blocks, H, 64, D] fp32 -> E4M3 codes as float8 and power-of-two scales [blocks, H]."""
    s = _pow2_scale(x.abs().amax(dim=(2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def _filled_cache(blocks, H, D, g):
    """A pool whose every block holds keys with a few strong channels and values of uneven heads."""
    kq = torch.empty(blocks, H, D // 64, BLOCK, 64, dtype=torch.uint8, device="cuda")
    vq = torch.empty(blocks, H, D, BLOCK, dtype=torch.uint8, device="cuda")
    ks = torch.empty(blocks, H, device="cuda")
    vs = torch.empty(blocks, H, device="cuda")
    chan = torch.ones(H, 1, D, device="cuda")
    chan[:, :, ::37] = 6.0
    head = torch.rand(H, 1, 1, generator=g, device="cuda") * 2 + 0.2
    step = max(1, (1 << 27) // (H * BLOCK * D))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        q, ks[i:i + n] = _quantised(torch.randn(n, H, BLOCK, D, generator=g, device="cuda") * chan)
        kq[i:i + n] = q.view(torch.uint8).view(n, H, BLOCK, D // 64, 64).transpose(2, 3)
        q, vs[i:i + n] = _quantised(torch.randn(n, H, BLOCK, D, generator=g, device="cuda") * head)
        vq[i:i + n] = q.view(torch.uint8).transpose(2, 3)
    return kq, vq, ks, vs


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op in ("append", "attn"):
        B, H, D = case["B"], case["H"], case["D"]
        st["table"], blocks = _table(case, g)
        st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        st["kq"], st["vq"], st["ks"], st["vs"] = _filled_cache(blocks, H, D, g)
    if op == "append":
        # new tokens of varying size: some blocks' scales have to grow, some stay
        size = torch.exp(torch.randn(case["B"], case["N"], 1, 1, generator=g, device="cuda") * 0.5)
        st["k"] = (torch.randn(B, case["N"], H, D, generator=g, device="cuda") * size * 2).bfloat16()
        st["v"] = (torch.randn(B, case["N"], H, D, generator=g, device="cuda") * size).bfloat16()
    elif op == "attn":
        q = torch.randn(B, case["M"], H * case["G"], D, generator=g, device="cuda")
        q[..., ::37] *= 0.3
        st["q"] = (q * 1.5).bfloat16()
        st["scale"] = 1.0 / math.sqrt(D)
    elif op == "logprobs":
        N, V = case["N"], case["V"]
        z = torch.randn(N, V, generator=g, device="cuda") * 2.5
        # a few tokens stand out, as a trained model's do; some words are masked away
        pick = torch.randint(0, V, (N, 24), generator=g, device="cuda")
        z.scatter_add_(1, pick, torch.rand(N, 24, generator=g, device="cuda") * 12)
        z[:, V // 2:V // 2 + V // 50] = float("-inf")
        st["z"] = z.to(getattr(torch, case["dtype"]))
        st["tokens"] = pick[:, 0].to(torch.int32).contiguous()
    else:
        N, V = case["N"], case["V"]
        emb = torch.empty(V, HIDDEN, dtype=torch.bfloat16, device="cuda")
        for i in range(0, V, 1 << 16):
            n = min(1 << 16, V - i)
            emb[i:i + n] = (torch.randn(n, HIDDEN, generator=g, device="cuda") * 0.02).bfloat16()
        # each row speaks for a dozen words with falling strength, over a floor of noise
        pick = torch.randint(0, V, (N, 12), generator=g, device="cuda")
        h = torch.randn(N, HIDDEN, generator=g, device="cuda") * 0.4
        for i in range(12):
            h += (9.0 - 0.9 * i) / 1.126 * emb[pick[:, i]].float()
        st["emb"], st["h"] = emb, h.bfloat16()
        st["tokens"] = pick[:, 1].to(torch.int32).contiguous()
    if own:
        import fine_grained_moe_gb300 as fgm
        if op in ("append", "attn"):
            st["cache"] = fgm.KVCache(st["kq"], st["vq"], st["ks"], st["vs"])
        if op == "attn":
            st["ws"] = fgm.Workspace("cuda", nbytes=fgm.attn_workspace_bytes(B, case["M"], H * case["G"], H, D))
        elif op == "append":
            st["ws"] = fgm.Workspace("cuda")
        elif op == "logprobs":
            st["ws"] = fgm.Workspace("cuda", nbytes=fgm.logprobs_workspace_bytes(N, V, case["k"]))
        else:
            st["ws"] = fgm.Workspace("cuda", nbytes=fgm.lm_head_logprobs_workspace_bytes(N, V, case["k"]))
    return st


# ---------------------------------------------------------------- plain forms
def _pow2_scale(amax):
    """Smallest power of two s with amax / s <= 448, at least MIN_SCALE."""
    m, e = torch.frexp(amax)     # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    s = (e - 9 + (m > 0.875).to(e.dtype) + 127).clamp(1, 254).to(torch.int32).__lshift__(23).view(torch.float32)
    return torch.where(amax > 0, s, torch.zeros_like(s)).clamp_min(MIN_SCALE)


def _append_side(codes, scales, phys, new, is_new, is_kept):
    """codes [B, nb, 64, H, D] uint8 of the touched blocks and new [.., H, D] fp32 -> their codes and scales."""
    old_s = scales[phys]                                                          # [B, nb, H]
    amax = torch.where(is_new[..., None, None], new.abs(), torch.zeros_like(new)).amax(dim=(2, 4))
    s = _pow2_scale(amax)
    s = torch.where(is_kept.any(dim=2)[..., None], torch.maximum(s, old_s), s)
    q_new = (new / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    kept = codes.view(torch.float8_e4m3fn).float() * (old_s / s)[:, :, None, :, None]
    q_kept = kept.to(torch.float8_e4m3fn).view(torch.uint8)
    out = torch.where(is_kept[..., None, None], q_kept, codes)
    return torch.where(is_new[..., None, None], q_new, out), s


def _append_plain(st):
    c = st["case"]
    B, N, H, D = c["B"], c["N"], c["H"], c["D"]
    lens = st["lens"].long()
    start = lens - N
    nb = (N + BLOCK - 2) // BLOCK + 1
    j = torch.minimum(start[:, None] // BLOCK + torch.arange(nb, device="cuda"), (lens[:, None] - 1) // BLOCK)
    tok = j[:, :, None] * BLOCK + torch.arange(BLOCK, device="cuda")               # [B, nb, 64]
    idx = tok - start[:, None, None]
    is_new, is_kept = (idx >= 0) & (idx < N), idx < 0
    phys = torch.gather(st["table"].long(), 1, j)
    row = torch.arange(B, device="cuda")[:, None, None]
    at = idx.clamp(0, N - 1)
    kc = st["kq"][phys].permute(0, 1, 4, 2, 3, 5).reshape(B, nb, BLOCK, H, D)
    kc, ks = _append_side(kc, st["ks"], phys, st["k"].float()[row, at], is_new, is_kept)
    st["kq"][phys] = kc.view(B, nb, BLOCK, H, D // 64, 64).permute(0, 1, 3, 4, 2, 5)
    st["ks"][phys] = ks
    vc = st["vq"][phys].permute(0, 1, 4, 2, 3)
    vc, vs = _append_side(vc, st["vs"], phys, st["v"].float()[row, at], is_new, is_kept)
    st["vq"][phys] = vc.permute(0, 1, 3, 4, 2)
    st["vs"][phys] = vs


def _attn_plain(st):
    c = st["case"]
    B, M, H, G, D, W = c["B"], c["M"], c["H"], c["G"], c["D"], c["window"]
    lens = st["lens"].long()
    per = st["table"].shape[1]
    nb = per if not W else min(per, (W + M + BLOCK - 3) // BLOCK + 1)
    first = torch.zeros_like(lens) if not W else (lens - M - W + 1).clamp_min(0) // BLOCK
    j = first[:, None] + torch.arange(nb, device="cuda")
    phys = torch.gather(st["table"].long(), 1, j.clamp_max(per - 1))
    T = nb * BLOCK
    t = (j[:, :, None] * BLOCK + torch.arange(BLOCK, device="cuda")).view(B, T)
    k = st["kq"][phys].view(torch.float8_e4m3fn).float() * st["ks"][phys][..., None, None, None]
    k = k.permute(0, 2, 1, 4, 3, 5).reshape(B, H, T, D)
    v = st["vq"][phys].view(torch.float8_e4m3fn).float() * st["vs"][phys][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(B, H, T, D)
    q = st["q"].float().view(B, M, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, M * G, D)
    s = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    pos = lens[:, None] - M + torch.arange(M, device="cuda")                       # [B, M]
    see = (t[:, None, :] <= pos[:, :, None]) & (t[:, None, :] < lens[:, None, None])
    if W:
        see = see & (t[:, None, :] > pos[:, :, None] - W)
    see = see[:, None, :, None, :].expand(B, H, M, G, T).reshape(B, H, M * G, T)
    s = torch.where(see, s, torch.full_like(s, float("-inf")))
    m = s.amax(dim=3, keepdim=True)
    e = torch.exp(s - m)
    l = e.sum(dim=3, keepdim=True)
    o = torch.matmul(e / l, v)
    lse = (m + torch.log(l))[..., 0]
    o = o.view(B, H, M, G, D).permute(0, 2, 1, 3, 4).reshape(B, M, H * G, D)
    return o.bfloat16(), lse.view(B, H, M, G).permute(0, 2, 1, 3).reshape(B, M, H * G).contiguous()


def _top_plain(x, k):
    """The k largest of each row, ties to the lower index: keys of value then index in 64 bits."""
    bits = x.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = order * (1 << 32) + (x.shape[1] - 1 - torch.arange(x.shape[1], device=x.device))
    return torch.topk(key, k, dim=1).indices


def _logprobs_plain(z, tokens, k, T):
    z = z.float()
    x = z / T
    m = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - m)
    l = e.sum(dim=1, keepdim=True)
    lse = m + torch.log(l)
    logp = x.gather(1, tokens.long()[:, None]) - lse
    mean = torch.where(e > 0, e * (x - m), torch.zeros_like(e)).sum(dim=1, keepdim=True) / l
    entropy = torch.log(l) - mean
    out = [logp[:, 0], entropy[:, 0]]
    if k:
        ids = _top_plain(z, k)
        out += [ids.to(torch.int32), x.gather(1, ids) - lse]
    return out


def run(st):
    c = st["case"]
    op = c["op"]
    if op == "append":
        if own:
            import fine_grained_moe_gb300 as fgm
            fgm.kv_append(st["cache"], st["k"], st["v"], st["lens"], block_table=st["table"], ws=st["ws"])
        else:
            _append_plain(st)
        # the codes as the E4M3 values they stand for
        return [st["kq"].view(torch.float8_e4m3fn), st["vq"].view(torch.float8_e4m3fn), st["ks"], st["vs"]]
    if op == "attn":
        if own:
            import fine_grained_moe_gb300 as fgm
            lse = torch.empty(c["B"], c["M"], c["H"] * c["G"], device="cuda")
            out = fgm.attn_fwd(st["cache"], st["q"], st["lens"], st["scale"], block_table=st["table"],
                               window=c["window"], lse=lse, ws=st["ws"])
            return [out, lse]
        return list(_attn_plain(st))
    if op == "logprobs":
        if own:
            import fine_grained_moe_gb300 as fgm
            r = fgm.logprobs(st["z"], st["tokens"], k=c["k"], T=c["T"], ws=st["ws"])
            return [x for x in (r.logp, r.entropy, r.top_ids, r.top_logp) if x is not None]
        return _logprobs_plain(st["z"], st["tokens"], c["k"], c["T"])
    if own:
        import fine_grained_moe_gb300 as fgm
        r = fgm.lm_head_logprobs(st["emb"], st["h"], st["tokens"], k=c["k"], T=c["T"], ws=st["ws"])
        return [x for x in (r.logp, r.entropy, r.top_ids, r.top_logp) if x is not None]
    z = torch.matmul(st["h"].float(), st["emb"].float().t())
    return _logprobs_plain(z, st["tokens"], c["k"], c["T"])


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "append":
        n = case["B"] * case["N"] * case["H"] * case["D"]
        blocks = sum((L - 1) // BLOCK - (L - case["N"]) // BLOCK + 1 for L in _lens(case))
        return {"bytes": 2 * n * 2 + 2 * n + 8 * blocks * case["H"], "flops": 2 * 3 * n}
    if op == "attn":
        M, H, G, D, W = case["M"], case["H"], case["G"], case["D"], case["window"]
        seen = pairs = 0
        for L in _lens(case):
            lo = max(0, L - M - W + 1) if W else 0
            seen += L - lo
            pairs += sum(L - M + i + 1 - (max(0, L - M + i - W + 1) if W else 0) for i in range(M) if L - M + i >= 0)
        rows = case["B"] * M * H * G
        return {"bytes": seen * H * 2 * D + 8 * H * (seen // BLOCK + case["B"]) + rows * (4 * D + 4),
                "flops": 4 * pairs * H * G * D}
    N, V = case["N"], case["V"]
    out = N * (12 + 8 * case["k"])
    if op == "logprobs":
        return {"bytes": N * V * (4 if case["dtype"] == "float32" else 2) + out, "flops": 7 * N * V}
    return {"bytes": 2 * HIDDEN * (V + N) + out, "flops": (2 * HIDDEN + 7) * N * V}


# ---------------------------------------------------------------- 64 bits
def _exact_append(st):
    """Token by token: the scale of each touched block from its new tokens and, where older ones stay, its old scale."""
    c = st["case"]
    B, N, H, D = c["B"], c["N"], c["H"], c["D"]

    def side(q, scales, x, token_dim_last):
        val = q.view(torch.float8_e4m3fn).double()
        if not token_dim_last:                       # K: [blocks, H, D/64, 64, 64] -> [blocks, H, 64, D]
            val = val.transpose(2, 3).reshape(val.shape[0], H, BLOCK, D)
        else:
            val = val.transpose(2, 3).contiguous()
        scl = scales.double()
        for b in range(B):
            L = lens[b]
            p0 = L - N
            while p0 < L:
                j, lo = p0 // BLOCK, p0 % BLOCK
                hi = min(BLOCK, lo + L - p0)
                blk = int(tab[b][j])
                new = x[b, p0 - (L - N):p0 - (L - N) + hi - lo].double().transpose(0, 1)      # [H, n, D]
                ratio = new.abs().amax(dim=(1, 2)) / E4M3_MAX
                s = torch.tensor([2.0 ** e for e in range(-60, 121)], dtype=torch.float64, device="cuda")
                s = s[torch.searchsorted(s, ratio)]        # the first power of two that is not below the ratio
                if lo:
                    s = torch.maximum(s, scl[blk])
                    val[blk, :, :lo] *= (scl[blk] / s)[:, None, None]
                val[blk, :, lo:hi] = new / s[:, None, None]
                scl[blk] = s
                p0 += hi - lo
        if not token_dim_last:
            return val.view(-1, H, BLOCK, D // 64, 64).transpose(2, 3).contiguous(), scl
        return val.transpose(2, 3).contiguous(), scl

    tab, lens = st["table"].tolist(), _lens(c)
    k, ks = side(st["kq"], st["ks"], st["k"], False)
    v, vs = side(st["vq"], st["vs"], st["v"], True)
    return [k, v, ks, vs]


def _exact_attn(st):
    c = st["case"]
    B, M, H, G, D, W = c["B"], c["M"], c["H"], c["G"], c["D"], c["window"]
    out = torch.zeros(B, M, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, M, H * G), float("-inf"), dtype=torch.float64, device="cuda")
    lens = _lens(c)
    for b in range(B):
        L = lens[b]
        lo = max(0, L - M - W + 1) // BLOCK if W else 0
        blocks = st["table"][b, lo:(L + BLOCK - 1) // BLOCK].long()
        for h in range(H):
            k = st["kq"][blocks, h].view(torch.float8_e4m3fn).double() * st["ks"][blocks, h].double()[:, None, None, None]
            k = k.transpose(1, 2).reshape(-1, D)
            v = st["vq"][blocks, h].view(torch.float8_e4m3fn).double() * st["vs"][blocks, h].double()[:, None, None]
            v = v.transpose(1, 2).reshape(-1, D)
            for i in range(M):
                pos = L - M + i
                if pos < 0:
                    continue
                a = (max(0, pos - W + 1) if W else 0) - lo * BLOCK
                e = pos + 1 - lo * BLOCK
                s = st["q"][b, i, h * G:(h + 1) * G].double() @ k[a:e].t() * st["scale"]
                out[b, i, h * G:(h + 1) * G] = torch.softmax(s, dim=1) @ v[a:e]
                lse[b, i, h * G:(h + 1) * G] = torch.logsumexp(s, dim=1)
    return [out, lse]


def _exact_logprobs(logits_of, N, V, tokens, k, T):
    """logits_of(i, j): fp64 logits of rows i..j; rows in slices that fit."""
    parts = []
    step = max(1, (1 << 28) // V)
    for i in range(0, N, step):
        z = logits_of(i, min(N, i + step))
        lp = torch.log_softmax(z / T, dim=1)
        p = torch.exp(lp)
        part = [lp.gather(1, tokens[i:i + step].long()[:, None])[:, 0],
                -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(dim=1)]
        if k:
            ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
            part += [ids.to(torch.int32), lp.gather(1, ids)]
        parts.append(part)
    return [torch.cat(x) for x in zip(*parts)]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] == "attn":
        return _exact_attn(st)
    if case["op"] == "logprobs":
        return _exact_logprobs(lambda i, j: st["z"][i:j].double(), case["N"], case["V"], st["tokens"], case["k"], case["T"])
    emb = st["emb"]

    def logits(i, j):
        h = st["h"][i:j].double()
        return torch.cat([h @ emb[a:a + (1 << 15)].double().t() for a in range(0, case["V"], 1 << 15)], dim=1)
    return _exact_logprobs(logits, case["N"], case["V"], st["tokens"], case["k"], case["T"])
