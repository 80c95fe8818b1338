"""Plain 64-bit forms of the KV-cache and log-probability operators, on host
arrays; only the number formats come from the oracle."""

import numpy as np

import oracle

BLOCK = 64
MIN_SCALE = 2.0 ** -60


def pow2_scale(a: float) -> float:
    """Smallest power of two s with a / s <= 448, at least 2^-60."""
    s = MIN_SCALE
    while a / s > 448.0:
        s *= 2.0
    return s


def k_natural(k_q: np.ndarray) -> np.ndarray:
    """[blocks, H, D/64, 64, 64] codes -> [blocks, H, 64 tokens, D]."""
    n, h, c = k_q.shape[:3]
    return np.ascontiguousarray(k_q.transpose(0, 1, 3, 2, 4).reshape(n, h, BLOCK, c * 64))


def k_cached(nat: np.ndarray) -> np.ndarray:
    n, h, _, d = nat.shape
    return np.ascontiguousarray(nat.reshape(n, h, BLOCK, d // 64, 64).transpose(0, 1, 3, 2, 4))


def append_side(codes, scales, x, lens, table):
    """codes [blocks, H, 64 tokens, D] uint8 and scales [blocks, H], in place; x [B, N, H, D] fp64."""
    B, N, H = x.shape[:3]
    for b in range(B):
        for j in range((int(lens[b]) + BLOCK - 1) // BLOCK):
            toks = [t for t in range(max(0, lens[b] - N), lens[b]) if t // BLOCK == j]
            if not toks:
                continue
            blk, lo = table[b][j], toks[0] % BLOCK
            for h in range(H):
                new = x[b, toks[0] - (lens[b] - N):toks[-1] + 1 - (lens[b] - N), h]
                fin = np.abs(new[np.isfinite(new)])
                s = pow2_scale(fin.max() if fin.size else 0.0)
                if lo:
                    old = float(scales[blk, h])
                    s = max(s, old)
                    if s > old:
                        codes[blk, h, :lo] = oracle.e4m3_encode(oracle.e4m3_decode(codes[blk, h, :lo]) * (old / s))
                clipped = np.where(np.isnan(new), 0.0, np.clip(new / s, -448.0, 448.0))
                codes[blk, h, lo:lo + len(toks)] = oracle.e4m3_encode(clipped)
                scales[blk, h] = s


def attn(q, k_val, v_val, lens, table, scale, window):
    """q [B, M, Hq, D] fp64; k_val, v_val [blocks, H, 64, D] fp64 (scales applied).
    Returns out, lse and, for error bounds, A = sum_t P_t |v_t|, vmax = max |v_t|
    over what the row sees, and ds = sum of |q_d k_d| scale and qmax * sum |k|
    scale at their largest over the row's tokens."""
    B, M, Hq, D = q.shape
    H = k_val.shape[1]
    out = np.zeros((B, M, Hq, D))
    A, vmax = np.zeros_like(out), np.zeros_like(out)
    lse = np.full((B, M, Hq), -np.inf)
    dq, dk = np.zeros((B, M, Hq)), np.zeros((B, M, Hq))
    for b in range(B):
        L = int(lens[b])
        if L == 0:
            continue
        blocks = [table[b][j] for j in range((L + BLOCK - 1) // BLOCK)]
        for hq in range(Hq):
            h = hq // (Hq // H)
            k = k_val[blocks, h].reshape(-1, D)
            v = v_val[blocks, h].reshape(-1, D)
            for i in range(M):
                pos = L - M + i
                if pos < 0:
                    continue
                a = max(0, pos - window + 1) if window else 0
                kk, vv = k[a:pos + 1], v[a:pos + 1]
                s = kk @ q[b, i, hq] * scale
                m = s.max()
                e = np.exp(s - m)
                P = e / e.sum()
                out[b, i, hq] = P @ vv
                lse[b, i, hq] = m + np.log(e.sum())
                A[b, i, hq] = P @ np.abs(vv)
                vmax[b, i, hq] = np.abs(vv).max(axis=0)
                dq[b, i, hq] = (np.abs(kk) @ np.abs(q[b, i, hq])).max() * scale
                dk[b, i, hq] = np.abs(kk).sum(axis=1).max() * np.abs(q[b, i, hq]).max() * scale
    return out, lse, A, vmax, dq, dk


def logprobs(z, tokens, k, T):
    """z [N, V] fp64 (NaN counts as -inf). Returns logp, entropy, top ids, top logp."""
    z = np.where(np.isnan(z), -np.inf, z)
    m = z.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore", over="ignore"):
        x = (z - m) / T
        e = np.exp(x)
        l = e.sum(axis=1, keepdims=True)
        lp = x - np.log(l)
        ent = np.log(l)[:, 0] - np.where(e > 0, e * x, 0).sum(axis=1) / l[:, 0]
    bad = ~np.isfinite(m[:, 0])
    lp[bad], ent[bad] = np.nan, np.nan
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k]
    V = z.shape[1]
    tok = np.asarray(tokens)
    inside = (tok >= 0) & (tok < V)
    got = np.where(inside, np.take_along_axis(lp, np.where(inside, tok, 0)[:, None], 1)[:, 0], -np.inf)
    got[bad] = np.nan
    return got, ent, ids, np.take_along_axis(lp, ids, 1)
