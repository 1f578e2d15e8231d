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
    """((dq, dk, dv), bounds) of sum(dout * out).  The bounds count the roundings of a backward
    that holds P and dS in bf16 (8 significant bits: spacing 2^-7 of the leading bit, so a
    rounding is off by up to 2^-8 of the value; dS carries P's and its own; P on its way to dv may
    be rounded to fp16 first, 2^-11 more), takes D from a bf16
    out (2^-8 of each |dout out|) and forms scores in fp32 (d + 8 roundings of the sum of |q k|): elementwise
    limits before the results' own rounding."""
    q, k, v, dout = (np.asarray(t, np.float64) for t in (q, k, v, dout))
    B, Hq, N, d = q.shape
    g = Hq // k.shape[1]
    ok = visible(np.arange(N), np.arange(N), window, sinks)
    got = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    lim = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    for b in range(B):
        for h in range(Hq):
            qq, kk, vv, do = q[b, h], k[b, h // g], v[b, h // g], dout[b, h]
            p, _ = softmax_rows(scale * (qq @ kk.T), ok)
            dp = do @ vv.T
            D = (p * dp).sum(-1, keepdims=True)
            ds = p * (dp - D)
            got[0][b, h] = scale * ds @ kk
            got[1][b, h // g] += scale * ds.T @ qq
            got[2][b, h // g] += p.T @ do
            slip = 2 * scale * (np.abs(qq) @ np.abs(kk).T) * (d + 8) * 2.0 ** -24 + 2.0 ** -18
            dp_mass = np.abs(do) @ np.abs(vv).T
            off = (np.abs(do) * (p @ np.abs(vv))).sum(-1, keepdims=True) * 2.0 ** -8
            e_ds = np.abs(ds) * (2.0 ** -7 + slip) + p * (off + (dp_mass + np.abs(D)) * d * 2.0 ** -24)
            lim[0][b, h] = scale * e_ds @ np.abs(kk)
            lim[1][b, h // g] += scale * e_ds.T @ np.abs(qq)
            lim[2][b, h // g] += (p * (2.0 ** -8 + 2.0 ** -11 + slip)).T @ np.abs(do)
    return got, lim


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
