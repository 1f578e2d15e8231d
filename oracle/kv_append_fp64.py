"""fp64 reference of the paged cache's write side (rotation, page mapping, E4M3 blocks).

Works on numpy copies: float caches (bf16 values widened), or E4M3 values (not codes) with
their scales.  Returned cache rows of new tokens are exact (fp64) values; the caller rounds.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -40


def rotate(x, positions, inv_freq, interleaved=False):
    """[T, H, d] rows rotated by their positions: pair i turns by positions * inv_freq[i]."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    half = len(inv_freq)
    if half == 0:
        return y
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def block_scale(amax):
    """The smallest power of two s >= 2^-40 with amax <= 448 s."""
    amax = np.asarray(amax, np.float64)
    m, e = np.frexp(amax / E4M3_MAX)
    s = np.ldexp(1.0, np.where(m == 0.5, e - 1, e))
    return np.where(amax > 0, np.maximum(s, SCALE_MIN), SCALE_MIN)


def e4m3(x):
    """Nearest E4M3 value (ties to even, magnitudes above 448 to 448) of fp64 numbers."""
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(x), E4M3_MAX)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(mag, 2.0 ** -6))), -6.0) - 3.0)
    return np.copysign(np.rint(mag / step) * step, x)


def new_tokens(seq_lens, cu_tokens):
    """(token row, sequence, position) of every new token."""
    rows = []
    for b, L in enumerate(seq_lens):
        t0, t1 = int(cu_tokens[b]), int(cu_tokens[b + 1])
        rows += [(t, b, int(L) - (t1 - t0) + (t - t0)) for t in range(t0, t1)]
    return rows


def append(x, cache, scale, block_table, seq_lens, cu_tokens):
    """One tensor (rotated keys, or values) into its cache: returns (cache, scale) as fp64
    copies.  ``cache`` [pages, H, page, d]: bf16 values with ``scale`` None, else E4M3 values
    with ``scale`` [pages, H, page / block]; new rows are x, or x / s before its rounding."""
    cache = np.array(cache, np.float64)
    page = cache.shape[2]
    by_block = {}
    block = page if scale is None else page // scale.shape[2]
    for t, b, pos in new_tokens(seq_lens, cu_tokens):
        phys = int(block_table[b][pos // page])
        by_block.setdefault((phys, pos % page // block), []).append((pos % page, t))
    scale = None if scale is None else np.array(scale, np.float64)
    for (phys, blk), rows in by_block.items():
        slots, ts = [r[0] for r in rows], [r[1] for r in rows]
        new = np.asarray(x, np.float64)[ts].transpose(1, 0, 2)      # [H, n, d]
        if scale is None:
            cache[phys][:, slots] = new
            continue
        amax = np.abs(new).max((1, 2))
        s, held = block_scale(amax), min(slots) - blk * block
        if held:
            old = scale[phys, :, blk]
            s = np.where(amax <= E4M3_MAX * old, old, s)
            part = slice(blk * block, blk * block + held)
            cache[phys][:, part] = e4m3(cache[phys][:, part] * (old / s)[:, None, None])
        scale[phys, :, blk] = s
        cache[phys][:, slots] = new / s[:, None, None]
    return cache, scale
