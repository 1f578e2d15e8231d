"""fp64 reference of sliding-window attention with sinks: forward, backward and paged decoding.

Query position i sees key j with j <= i and (j > i - window or j < sinks).  With window None
the mask is causal (or full, for decoding).  numpy only; every (batch, head) in a loop.
"""
from __future__ import annotations

import numpy as np


def visible(i, j, window, sinks):
    """Boolean mask [len(i), len(j)] of query positions i and key positions j."""
    i, j = np.asarray(i)[:, None], np.asarray(j)[None]
    ok = j <= i
    if window is not None:
        ok &= (j > i - window) | (j < sinks)
    return ok


def softmax_rows(x, ok):
    """(weights, lse) of scores x where ok; rows that see nothing: weights 0, lse -inf."""
    x = np.where(ok, x, -np.inf)
    m = x.max(-1, keepdims=True, initial=-np.inf)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(x - m)
    l = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[..., 0]
    return e / np.where(l > 0, l, 1.0), lse


def forward(q, k, v, scale, window, sinks, key_offset=0):
    """out [B, Hq, N, d], lse [B, Hq, N] and the weighted mean of |v| (for error bounds)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    B, Hq, N, d = q.shape
    g = Hq // k.shape[1]
    ok = visible(np.arange(N) + key_offset, np.arange(N), window, sinks)
    out, mean, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        for h in range(Hq):
            p, lse[b, h] = softmax_rows(scale * (q[b, h] @ k[b, h // g].T), ok)
            out[b, h], mean[b, h] = p @ v[b, h // g], p @ np.abs(v[b, h // g])
    return out, lse, mean


def backward(q, k, v, dout, scale, window, sinks):
    """(dq, dk, dv) of sum(dout * out)."""
    q, k, v, dout = (np.asarray(t, np.float64) for t in (q, k, v, dout))
    B, Hq, N, d = q.shape
    g = Hq // k.shape[1]
    ok = visible(np.arange(N), np.arange(N), window, sinks)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(B):
        for h in range(Hq):
            p, _ = softmax_rows(scale * (q[b, h] @ k[b, h // g].T), ok)
            dp = dout[b, h] @ v[b, h // g].T
            ds = p * (dp - (p * dp).sum(-1, keepdims=True))
            dq[b, h] = scale * ds @ k[b, h // g]
            dk[b, h // g] += scale * ds.T @ q[b, h]
            dv[b, h // g] += p.T @ dout[b, h]
    return dq, dk, dv


def decode(q, k_cache, v_cache, block_table, seq_lens, scale=None, mask="causal", window=None, sinks=0):
    """(out, lse, mean |v|, largest sum |q k| of a row) of a paged decoding step; the caches hold
    values.  Only positions that some row sees are looked up; a length of 0 is an idle slot."""
    q = np.asarray(q, np.float64)
    B, Hq, Nq, d = q.shape
    Hkv, page = k_cache.shape[1], k_cache.shape[2]
    g = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    out, mean = np.zeros(q.shape), np.zeros(q.shape)
    lse, mass = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    for b in range(B):
        L = int(seq_lens[b])
        if L == 0:
            continue
        i, j = np.arange(L - Nq, L), np.arange(L)
        if mask == "sliding_window":
            j = j[(j > L - Nq - window) | (j < sinks)]
        ok = np.ones((Nq, len(j)), bool) if mask == "full" else \
            visible(i, j, window if mask == "sliding_window" else None, sinks)
        phys = np.array([int(block_table[b][x // page]) for x in j])
        for hk in range(Hkv):
            kk = np.asarray(k_cache[phys, hk, j % page], np.float64)
            vv = np.asarray(v_cache[phys, hk, j % page], np.float64)
            for h in range(hk * g, hk * g + g):
                p, lse[b, h] = softmax_rows(scale * (q[b, h] @ kk.T), ok)
                out[b, h], mean[b, h] = p @ vv, p @ np.abs(vv)
                mass[b, h] = scale * np.where(ok, np.abs(q[b, h]) @ np.abs(kk).T, 0).max(-1, initial=0)
    return out, lse, mean, mass
