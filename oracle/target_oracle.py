"""fp64 CPU oracle of the target-side operators (append to the paged cache,
attention over it, token log probabilities).

TEST INFRASTRUCTURE ONLY, like ``dflash_oracle``: plain loops and numpy in
float64 from the stored inputs, sharing no code with the CUDA path.

Paged layout: K pages [page][kv head][slot][d], V pages [page][kv head][d][slot],
64 slots; position p of request b is slot p % 64 of page table[b][p // 64].
A page outside the pool holds nothing.
"""
from __future__ import annotations

import numpy as np

PAGE = 64


def head_norm_rope(x, gain, eps: float, base: float, pos: int) -> np.ndarray:
    """One head: y = g x / sqrt(mean x^2 + eps) (gain None: y = x), then the
    pairs (i, i + d/2) turned by pos * base^(-2i/d) (base 0: not turned)."""
    y = np.asarray(x, dtype=np.float64)
    if gain is not None:
        y = np.asarray(gain, dtype=np.float64) * y / np.sqrt(np.mean(y * y) + eps)
    if base == 0:
        return y
    half = y.shape[-1] // 2
    out = np.empty_like(y)
    for i in range(half):
        a = pos * float(base) ** (-2.0 * i / (2 * half))
        c, s = np.cos(a), np.sin(a)
        out[i] = y[i] * c - y[i + half] * s
        out[i + half] = y[i + half] * c + y[i] * s
    return out


def append(k, v, table, qkv, nq, nkv, d, g_q, g_k, eps, base, cu_new, ctx_len):
    """K and V pools of one layer (float64 copies, updated) and the rotated
    queries [tokens][nq d] (NaN where no request owns the row)."""
    k, v = np.array(k, dtype=np.float64), np.array(v, dtype=np.float64)
    q = np.full((qkv.shape[0], nq * d), np.nan)
    for b in range(len(ctx_len)):
        for t in range(cu_new[b], cu_new[b + 1]):
            pos = int(ctx_len[b]) + t - int(cu_new[b])
            row = np.asarray(qkv[t], dtype=np.float64)
            for h in range(nq):
                q[t, h * d:(h + 1) * d] = head_norm_rope(row[h * d:(h + 1) * d], g_q, eps, base, pos)
            page = int(table[b][pos // PAGE]) if pos // PAGE < len(table[b]) else -1
            if not 0 <= page < k.shape[0]:
                continue
            for h in range(nkv):
                o = (nq + h) * d
                k[page, h, pos % PAGE] = head_norm_rope(row[o:o + d], g_k, eps, base, pos)
                v[page, h, :, pos % PAGE] = row[o + nkv * d:o + (nkv + 1) * d]
    return k, v, q


def attend(k, v, table, q, nq, nkv, d, cu_new, ctx_len, window, scale):
    """(out, lse, spread): attention of each new token over the positions it
    sees, and sum_t p_t |v_t| (what roundings of the p_t scale with); rows that
    no request owns are NaN."""
    T = q.shape[0]
    out, lse, spread = (np.full(s, np.nan) for s in ((T, nq * d), (T, nq), (T, nq * d)))
    for b in range(len(ctx_len)):
        for t in range(cu_new[b], cu_new[b + 1]):
            pos = int(ctx_len[b]) + t - int(cu_new[b])
            lo = max(0, pos - window + 1) if window else 0
            seen = [p for p in range(lo, pos + 1) if 0 <= table[b][p // PAGE] < k.shape[0]]
            pages = np.array([table[b][p // PAGE] for p in seen], dtype=np.int64)
            slots = np.array([p % PAGE for p in seen], dtype=np.int64)
            for h in range(nq):
                cols = slice(h * d, (h + 1) * d)
                if not seen:
                    out[t, cols], lse[t, h], spread[t, cols] = 0.0, -np.inf, 0.0
                    continue
                kk = np.asarray(k[pages, h // (nq // nkv), slots], dtype=np.float64)
                vv = np.asarray(v[pages, h // (nq // nkv), :, slots], dtype=np.float64)
                s = scale * (kk @ np.asarray(q[t, cols], dtype=np.float64))
                m = s.max()
                e = np.exp(s - m)
                out[t, cols] = (e @ vv) / e.sum()
                spread[t, cols] = (e @ np.abs(vv)) / e.sum()
                lse[t, h] = m + np.log(e.sum())
    return out, lse, spread


def token_logprobs(x, token, temperature: float, n_top: int):
    """(logprob, entropy, rank, top ids, top logprobs) of one row of logits."""
    y = np.asarray(x, dtype=np.float64) / temperature
    V = len(y)
    order = sorted(range(V), key=lambda i: (-y[i], i))
    m = y.max()
    if m == -np.inf:
        lp, entropy = np.full(V, -np.inf), 0.0
    else:
        lp = y - m - np.log(np.exp(y - m).sum())
        p = np.exp(lp)
        entropy = -sum(p[i] * lp[i] for i in range(V) if p[i] > 0)
    return lp[token], entropy, order.index(token), order[:n_top], lp[order[:n_top]]
