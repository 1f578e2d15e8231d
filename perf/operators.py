"""Operators around the paged key/value cache and the sliding window, with their plain forms.

Three operators of serving and training with long contexts:

* ``append``: new tokens' keys and values, rotated by their positions, go into a paged cache
  (bf16, or E4M3 codes with a power-of-two scale for each block of tokens and head), and the
  rotated queries come back in the decoding step's layout;
* ``decode8``: a decoding step over a paged cache held in E4M3 codes with a scale for each
  block of tokens and head (optionally with a sliding window and sinks);
* ``sink_fwd`` / ``sink_bwd`` / ``sink_decode``: attention with a causal sliding window of
  which the first ``sinks`` positions stay visible: forward, backward, and a decoding step
  over a bf16 paged cache.

With ``own`` false, ``run`` computes them with elementary torch operations in fp32 (angles in
fp64), rounded once; with ``own`` true it calls the package.
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
THETA = 500000.0   # base of the rotation's frequencies (long-context setting)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One new token for each of 32 running sequences with 64k-128k positions behind them: the
        # append of every decoding step, where latency counts.
        dict(name="append_step", kind="append", B=32, Hq=32, Hkv=8, d=128, page=16, block=0, tokens=32, uniform=True,
             rot=128, interleaved=False, L=131072),
        # A prefill chunk of 16384 tokens, six sequences of different lengths, 64 query heads.
        dict(name="append_prefill", kind="append", B=6, Hq=64, Hkv=8, d=128, page=16, block=0, tokens=16384,
             uniform=False, rot=128, interleaved=False, L=32768),
        # A prefill chunk into an 8-bit cache; the first block of each sequence is partly filled.
        dict(name="append_kv8", kind="append", B=5, Hq=32, Hkv=8, d=128, page=64, block=16, tokens=8191,
             uniform=False, rot=128, interleaved=False, L=32768),
        # A few short chats: latency.
        dict(name="decode8_small", kind="decode8", B=4, Hq=8, Hkv=2, Nq=1, d=128, Lmin=1, Lmax=1000, page=16, block=16,
             window=0, sinks=0),
        # One 128k-token sequence, 64 query heads on 8 KV heads.
        dict(name="decode8_gqa", kind="decode8", B=1, Hq=64, Hkv=8, Nq=1, d=128, Lmin=131072, Lmax=131072, page=16,
             block=16, window=0, sinks=0),
        # A ragged batch without shared heads.
        dict(name="decode8_mha", kind="decode8", B=16, Hq=32, Hkv=32, Nq=1, d=128, Lmin=8192, Lmax=32768, page=16,
             block=16, window=0, sinks=0),
        # Four drafted tokens verified for each of eight sequences.
        dict(name="decode8_spec", kind="decode8", B=8, Hq=64, Hkv=8, Nq=4, d=128, Lmin=16384, Lmax=32768, page=64,
             block=64, window=0, sinks=0),
        # Streaming generation from an 8-bit cache: a 4096-token window and four sinks.
        dict(name="sink_decode8", kind="decode8", B=32, Hq=32, Hkv=8, Nq=1, d=128, Lmin=65536, Lmax=131072, page=64,
             block=64, window=4096, sinks=4),
        # The same over a bf16 cache.
        dict(name="sink_decode", kind="sink_decode", B=32, Hq=32, Hkv=8, Nq=1, d=128, Lmin=65536, Lmax=131072, page=16,
             window=4096, sinks=4),
        # Prefill or training forward of a long sequence.
        dict(name="sink_fwd", kind="sink_fwd", B=1, Hq=32, Hkv=8, N=32768, d=128, window=1024, sinks=16),
        # Training backward, shared heads.
        dict(name="sink_bwd", kind="sink_bwd", B=1, Hq=32, Hkv=8, N=16384, d=128, window=1024, sinks=4),
        # Training backward without shared heads, odd lengths, more sinks than a tile.
        dict(name="sink_bwd_mha", kind="sink_bwd", B=2, Hq=8, Hkv=8, N=5001, d=128, window=500, sinks=130),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "append", "decode8", "decode8", "decode8", "sink_fwd", "sink_bwd", "sink_decode"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "append":
        d = rng.choice([64, 128])
        B = _spread(rng, 1, 64)
        block = rng.choice([0, 0, 1, 16, 32, page])
        uniform = rng.random() < 0.5
        tokens = B * _spread(rng, 1, 8) if uniform else _spread(rng, 1, 16000)
        return dict(kind=kind, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, block=min(block, page), tokens=tokens,
                    uniform=uniform, rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3,
                    L=_spread(rng, 32, 131072))
    if kind in ("decode8", "sink_decode"):
        B = _spread(rng, 1, 32)
        Nq = rng.choice([1, 1, 1, 2, 3, 5, 8])
        Lmax = _spread(rng, 40, min(131072, 4000000 // (B * Hkv)))
        window, sinks = 0, 0
        if kind == "sink_decode" or rng.random() < 0.4:
            window, sinks = _spread(rng, 1, 8192), rng.choice([0, 1, 4, 64, 129, 300])
        if kind == "sink_decode":
            return dict(kind=kind, B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, d=rng.choice([64, 128]), Lmin=max(Nq, Lmax // 3),
                        Lmax=Lmax, page=page, window=window, sinks=max(1, sinks))
        return dict(kind=kind, B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, d=rng.choice([64, 128]), Lmin=max(Nq, Lmax // 3), Lmax=Lmax,
                    page=page, block=rng.choice([1, 16, page]), window=window, sinks=sinks)
    B = rng.choice([1, 1, 2])
    N = _spread(rng, 1, 12000) if kind == "sink_fwd" else _spread(rng, 9, 12000)   # one row alone has no dq, dk
    return dict(kind=kind, B=B, Hq=min(Hq, 4 * Hkv), Hkv=Hkv, N=N, d=rng.choice([64, 128]), window=_spread(rng, 1, 1200),
                sinks=rng.choice([1, 2, 4, 16, 100, 128, 200]))


# ------------------------------------------------------------------ inputs
def _scales(amax):
    """The power of two s with amax <= 448 s, at least 2^-40."""
    m, e = torch.frexp(amax.double() / 448.0)          # amax / 448 = m 2^e, 0.5 <= m < 1
    s = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))
    return torch.where(amax > 0, s, torch.zeros_like(s)).clamp_min(2.0 ** -40).float()


def _quantised(x, block):
    """E4M3 codes [P, H, page, d] and scales [P, H, page / block] of an fp32 pool."""
    P, H, page, d = x.shape
    xb = x.view(P, H, page // block, block * d)
    s = _scales(xb.abs().amax(-1))
    return (xb / s[..., None]).to(E4M3).view(P, H, page, d), s


def _pages(first, last, width, rs, device):
    """A page table: sequence b keeps logical pages first[b]..last[b], handed out in random order."""
    counts = np.maximum(last - first + 1, 0)
    perm = rs.permutation(int(counts.sum()))
    table, at = np.full((len(first), width), -1, np.int32), 0
    for b, n in enumerate(counts):
        table[b, first[b]:first[b] + n] = perm[at:at + n]
        at += int(n)
    return torch.from_numpy(table).to(device), int(counts.sum())


def prepare(case, seed):
    c, dev = case, "cuda"
    rs = np.random.RandomState((seed * 1000003 + 17) % (1 << 32))
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    s = dict(case=c)
    if c["kind"] == "append":
        B, T, ps, Hkv, Hq, d = c["B"], c["tokens"], c["page"], c["Hkv"], c["Hq"], c["d"]
        if c["uniform"]:
            n = np.full(B, T // B)
        else:
            cuts = np.sort(rs.randint(0, T + 1, B - 1))
            n = np.diff(np.concatenate([[0], cuts, [T]]))
        start = rs.randint(0, c["L"], B)
        L = start + n
        s["block_table"], _ = _pages(start // ps, np.where(n > 0, (L - 1) // ps, start // ps - 1),
                                     int((max(L.max(), 1) - 1) // ps) + 1, rs, dev)
        pool = T // ps + 2 * B      # the pages of the new tokens, and some that no table names
        # one projection's output, of which q, k and v are views
        qkv = randn(T, (Hq + 2 * Hkv) * d)
        qkv[:, Hq * d:] *= torch.exp(0.7 * torch.randn((T, 1), generator=g, device=dev)).bfloat16()
        s["q"] = qkv[:, :Hq * d].view(T, Hq, d)
        s["k"] = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
        s["v"] = qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
        s["seq_lens"] = torch.from_numpy(L.astype(np.int32)).to(dev)
        s["cu_tokens"] = None if c["uniform"] else torch.from_numpy(
            np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(dev)
        s["inv_freq"] = (THETA ** (-torch.arange(c["rot"] // 2, device=dev, dtype=torch.float64) * 2 / c["rot"])).float()
        for name in ("k", "v"):
            x = randn(pool, Hkv, ps, d, dtype=torch.float32)
            if c["block"]:
                s[name + "_cache"], s[name + "_scale"] = _quantised(x, c["block"])
            else:
                s[name + "_cache"], s[name + "_scale"] = x.bfloat16(), None
        return s
    if c["kind"] in ("decode8", "sink_decode"):
        B, ps, Hkv, d = c["B"], c["page"], c["Hkv"], c["d"]
        L = rs.randint(c["Lmin"], c["Lmax"] + 1, B)
        first = np.zeros(B, np.int64)
        if c["window"]:      # pages behind the window are recycled, but for the sinks'
            first = np.maximum(L - c["Nq"] - c["window"] + 1, 0) // ps
            keep = np.minimum((min(c["sinks"], int(L.max())) + ps - 1) // ps, first)
        last = (L - 1) // ps
        width = int(last.max()) + 1
        table, pool = _pages(first, last, width, rs, dev)
        if c["window"] and keep.any():
            more, sunk = _pages(np.zeros(B, np.int64), keep - 1, width, rs, dev)
            table = torch.where(more >= 0, more + pool, table)
            pool += sunk
        s["q"], s["block_table"] = randn(B, c["Hq"], c["Nq"], d), table
        s["seq_lens"], s["max_len"] = torch.from_numpy(L.astype(np.int32)).to(dev), int(L.max())
        for name in ("k", "v"):
            x = randn(pool, Hkv, ps, d, dtype=torch.float32 if c["kind"] == "decode8" else torch.bfloat16)
            if c["kind"] == "decode8":   # blocks of different magnitudes
                xb = x.view(pool, Hkv, ps // c["block"], -1)
                xb *= torch.exp(0.5 * torch.randn(xb.shape[:3] + (1,), generator=g, device=dev))
                x, s[name + "_scale"] = _quantised(x, c["block"])
            s[name + "_cache"] = x
        return s
    B, N, d = c["B"], c["N"], c["d"]
    s["q"], s["k"], s["v"] = randn(B, c["Hq"], N, d), randn(B, c["Hkv"], N, d), randn(B, c["Hkv"], N, d)
    if c["kind"] == "sink_bwd":          # the forward's outputs, which a training step has by then
        s["dout"] = randn(B, c["Hq"], N, d)
        s["out"], s["lse"] = _sink_fwd(s)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"append": _own_append, "decode8": _own_decode8, "sink_decode": _own_sink_decode,
                "sink_fwd": _own_sink_fwd, "sink_bwd": _own_sink_bwd}[kind](state)
    return {"append": _append, "decode8": _decode, "sink_decode": _decode, "sink_fwd": _sink_fwd,
            "sink_bwd": _sink_bwd}[kind](state)


def _package():
    import exact_io_aware_72_b200 as attn
    return attn


def _own_append(s):
    attn = _package()
    q = attn.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], q=s["q"],
                       cu_tokens=s["cu_tokens"], inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"],
                       k_scale=s["k_scale"], v_scale=s["v_scale"])
    out = dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
    if s["case"]["block"]:
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def _own_decode8(s):
    attn, c = _package(), s["case"]
    mask, window = ("sliding_window", c["window"]) if c["window"] else ("causal", None)
    if "plan" not in s:      # split count and workspace, kept by a program from step to step
        n = attn.decode_kv8_num_splits(c["B"], c["Hq"], c["Hkv"], c["Nq"], s["max_len"], mask, window, c["sinks"])
        s["plan"] = n, attn.decode_kv8_workspace(c["B"], c["Hq"], c["Hkv"], c["Nq"], c["d"], n, device=s["q"].device)
    return attn.decode_kv8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                           s["seq_lens"], mask=mask, window=window, sinks=c["sinks"], num_splits=s["plan"][0],
                           workspace=s["plan"][1])


def _own_sink_decode(s):
    attn, c = _package(), s["case"]
    if "plan" not in s:
        n = attn.decode_num_splits(c["B"], c["Hq"], c["Hkv"], c["Nq"], s["max_len"], "sliding_window", c["window"])
        s["plan"] = n, torch.zeros(attn.decode_workspace_bytes(c["B"], c["Hq"], c["Nq"], c["d"], n) // 4,
                                   device=s["q"].device)
    return attn.decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], mask="sliding_window",
                       window=c["window"], sinks=c["sinks"], num_splits=s["plan"][0], workspace=s["plan"][1])


def _own_sink_fwd(s):
    c = s["case"]
    return _package().fwd(s["q"], s["k"], s["v"], mask="sliding_window", window=c["window"], sinks=c["sinks"])


def _own_sink_bwd(s):
    c = s["case"]
    return _package().bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], mask="sliding_window",
                          window=c["window"], sinks=c["sinks"])


# ------------------------------------------------------------------ plain forms
def _rotated(x, cos, sin, interleaved):
    """fp32 rotation of [T, H, d]: pairs (i, i + rot / 2), or (2i, 2i + 1)."""
    x, half = x.float(), cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., 2 * half:]], -1)


def _append(s):
    c, table = s["case"], s["block_table"]
    B, T, ps = c["B"], c["tokens"], c["page"]
    L = s["seq_lens"].long()
    cu = s["cu_tokens"].long() if s["cu_tokens"] is not None else \
        torch.arange(B + 1, device=L.device) * (T // B)
    t = torch.arange(T, device=L.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = L[b] - cu[b + 1] + t
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotated(s["q"], cos, sin, c["interleaved"]).bfloat16()
    if s["cu_tokens"] is None:
        q = q.view(B, T // B, c["Hq"], c["d"]).transpose(1, 2).contiguous()
    k, v = _rotated(s["k"], cos, sin, c["interleaved"]), s["v"].float()
    page, slot = table[b, pos // ps].long(), pos % ps
    out = dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
    if not c["block"]:
        s["k_cache"][page, :, slot] = k.bfloat16()
        s["v_cache"][page, :, slot] = v.bfloat16()
        return out
    for name, x in (("k", k), ("v", v)):
        _append8(s[name + "_cache"], s[name + "_scale"], x, page, slot, L, cu, table, c)
    out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def _append8(cache, scale, x, page, slot, L, cu, table, c):
    """Quantise rows x [T, H, d] into blocks of `block` slots. A block that starts with a new
    token takes the scale of its new tokens. One that held tokens before keeps its scale where
    the new ones fit, and otherwise takes theirs, its older codes being rounded again."""
    ps, bs, H, d = c["page"], c["block"], c["Hkv"], c["d"]
    P, nb = cache.shape[0], ps // bs
    amax = torch.zeros(P * nb, H, device=x.device)
    at = page * nb + slot // bs
    amax.scatter_reduce_(0, at[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    old = scale.view(P, H, nb).transpose(1, 2).reshape(P * nb, H)
    n = cu[1:] - cu[:-1]
    first = (L - n).clamp_min(0)
    held = (first % bs) * (n > 0)                          # slots of the first block filled before
    fp = table.gather(1, (first // ps).clamp_max(table.shape[1] - 1)[:, None])[:, 0].long().clamp_min(0)
    part = torch.zeros(P * nb, device=x.device, dtype=torch.int64)
    part.scatter_reduce_(0, fp * nb + first % ps // bs, held, "amax")
    fresh = _scales(amax)
    new = torch.where((part > 0)[:, None] & (amax <= 448.0 * old), old, fresh)
    touched = torch.zeros(P * nb, device=x.device, dtype=torch.bool)
    touched[at] = True
    new = torch.where(touched[:, None], new, old)
    # older codes of the partly filled blocks, under the new scale
    ratio = (old / new).view(P, nb, H).transpose(1, 2)
    rows = (part.view(P, 1, nb, 1) > torch.arange(bs, device=x.device)) & (ratio != 1)[..., None]
    codes = cache.view(P, H, nb, bs, d)
    again = (codes.float() * ratio[..., None, None]).to(E4M3)
    codes.view(torch.uint8).copy_(torch.where(rows[..., None], again.view(torch.uint8), codes.view(torch.uint8)))
    scale.copy_(new.view(P, nb, H).transpose(1, 2))
    cache.view(torch.uint8)[page, :, slot] = (x / new[at][..., None]).to(E4M3).view(torch.uint8)


def _decode(s):
    c = s["case"]
    B, Hkv, Nq, d, ps = c["B"], c["Hkv"], c["Nq"], c["d"], c["page"]
    L, dev = s["seq_lens"].long(), s["q"].device
    w, sinks = c["window"], c["sinks"]
    if w:
        near = torch.arange(min(w + Nq - 1, s["max_len"]), device=dev)
        near = L[:, None] - near.numel() + near
        far = torch.arange(min(sinks, s["max_len"]), device=dev).expand(B, -1)
        pos = torch.cat([torch.where(far < near[:, :1], far, -1), near], 1)
    else:
        pos = torch.arange(s["max_len"], device=dev).expand(B, -1)
    qpos = L[:, None, None] - Nq + torch.arange(Nq, device=dev)[:, None]
    seen = (pos >= 0)[:, None] & (pos[:, None] <= qpos)
    if w:
        seen &= (pos[:, None] > qpos - w) | (pos[:, None] < sinks)
    p = pos.clamp_min(0)
    page, slot = s["block_table"].gather(1, p // ps).long().clamp_min(0), p % ps
    k, v = s["k_cache"][page, :, slot].float(), s["v_cache"][page, :, slot].float()   # [B, M, Hkv, d]
    if c["kind"] == "decode8":
        k = k * s["k_scale"][page, :, slot // c["block"]][..., None]
        v = v * s["v_scale"][page, :, slot // c["block"]][..., None]
    q = s["q"].float().view(B, Hkv, -1, d)
    S = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, Hkv, -1, Nq, pos.shape[1]) / math.sqrt(d)
    S = S.masked_fill(~seen[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    e = (S - m).exp()
    l = e.sum(-1, keepdim=True)
    out = torch.matmul(e.view(B, Hkv, -1, pos.shape[1]), v.transpose(1, 2)).view(B, Hkv, -1, Nq, d) / l
    return out.reshape(B, c["Hq"], Nq, d).bfloat16(), (m + l.log()).reshape(B, c["Hq"], Nq)


def _bands(s):
    """The window as chunks of C queries against 2 C keys (their own chunk and the one before),
    and the sinks beside them: chunked tensors and the two masks."""
    c = s["case"]
    N, w = c["N"], c["window"]
    C = min(N, max(w, 64))
    n, S = -(-N // C), min(c["sinks"], N)
    i = torch.arange(n * C, device=s["q"].device).view(n, C, 1)
    j = i[:, :1] - C + torch.arange(2 * C, device=s["q"].device)
    band = (j >= 0) & (j < N) & (j <= i) & (j > i - w)
    j = torch.arange(S, device=s["q"].device)
    return C, n, S, band, (j <= i - w)


def _chunks(x, C, n, heads):
    """[B, H, N, d] to fp32 [B, heads, H / heads, n, C, d], zeros behind the last row."""
    B, H, N, d = x.shape
    x = torch.cat([x.float(), x.new_zeros((B, H, n * C - N, d), dtype=torch.float32)], 2)
    return x.view(B, heads, H // heads, n, C, d)


def _pairs(x):
    """Chunks [B, H, 1, n, C, d] to [B, H, 1, n, 2 C, d]: the chunk before each, and itself."""
    return torch.cat([torch.cat([torch.zeros_like(x[:, :, :, :1]), x[:, :, :, :-1]], 3), x], 4)


def _sink_scores(s):
    c = s["case"]
    C, n, S, band, far = _bands(s)
    q, k = _chunks(s["q"], C, n, c["Hkv"]), _chunks(s["k"], C, n, c["Hkv"])
    sink = s["k"][:, :, None, None, :S].float()
    near = torch.matmul(q, _pairs(k).transpose(-1, -2)).mul_(1 / math.sqrt(c["d"])).masked_fill_(~band, -math.inf)
    away = torch.matmul(q, sink.transpose(-1, -2)).mul_(1 / math.sqrt(c["d"])).masked_fill_(~far, -math.inf)
    return C, n, S, q, k, sink, near, away


def _sink_fwd(s):
    c = s["case"]
    C, n, S, q, k, sink, near, away = _sink_scores(s)
    m = torch.maximum(near.amax(-1, keepdim=True), away.amax(-1, keepdim=True)).clamp_min(-1e30)
    near, away = near.sub_(m).exp_(), away.sub_(m).exp_()
    l = near.sum(-1, keepdim=True) + away.sum(-1, keepdim=True)
    out = torch.matmul(near, _pairs(_chunks(s["v"], C, n, c["Hkv"])))
    out = (out + torch.matmul(away, s["v"][:, :, None, None, :S].float())) / l
    out = out.reshape(c["B"], c["Hq"], n * C, c["d"])[:, :, :c["N"]].bfloat16().contiguous()
    return out, (m + l.log()).reshape(c["B"], c["Hq"], n * C)[:, :, :c["N"]].contiguous()


def _sink_bwd(s):
    c = s["case"]
    B, Hkv, N, d = c["B"], c["Hkv"], c["N"], c["d"]
    C, n, S, q, k, sink, near, away = _sink_scores(s)
    lse = _chunks(s["lse"][..., None], C, n, Hkv)
    do, v = _chunks(s["dout"], C, n, Hkv), _chunks(s["v"], C, n, Hkv)
    delta = (do * _chunks(s["out"], C, n, Hkv)).sum(-1, keepdim=True)
    vs = s["v"][:, :, None, None, :S].float()
    near, away = near.sub_(lse).exp_(), away.sub_(lse).exp_()
    dv, dvs = torch.matmul(near.transpose(-1, -2), do).sum(2), torch.matmul(away.transpose(-1, -2), do).sum((2, 3))
    near *= torch.matmul(do, _pairs(v).transpose(-1, -2)).sub_(delta)
    away *= torch.matmul(do, vs.transpose(-1, -2)).sub_(delta)
    near *= 1 / math.sqrt(d)
    away *= 1 / math.sqrt(d)
    dq = torch.matmul(near, _pairs(k)) + torch.matmul(away, sink)
    dk, dks = torch.matmul(near.transpose(-1, -2), q).sum(2), torch.matmul(away.transpose(-1, -2), q).sum((2, 3))

    def joined(x, xs):      # a chunk's rows: from its own queries, from the next chunk's, and as sinks
        y = x[:, :, :, C:].clone()
        y[:, :, :-1] += x[:, :, 1:, :C]
        y = y.reshape(B, Hkv, n * C, d)[:, :, :N].clone()
        y[:, :, :S] += xs
        return y.bfloat16()

    return dq.reshape(B, c["Hq"], n * C, d)[:, :, :N].bfloat16().contiguous(), joined(dk, dks), joined(dv, dvs)


# ------------------------------------------------------------------ work
def work(case):
    c = case
    if c["kind"] == "append":
        rows, width = c["tokens"], 1 if c["block"] else 2
        moved = rows * c["d"] * ((c["Hq"] + 2 * c["Hkv"]) * 2 + c["Hq"] * 2 + 2 * c["Hkv"] * width)
        if c["block"]:
            moved += 2 * c["Hkv"] * (rows // c["block"] + c["B"]) * 4
        return dict(bytes=moved, flops=3 * rows * c["rot"] * (c["Hq"] + c["Hkv"]))
    if c["kind"] in ("decode8", "sink_decode"):
        keys = (c["Lmin"] + c["Lmax"]) / 2
        if c["window"]:
            keys = min(keys, c["window"] + c["Nq"] - 1 + c["sinks"])
        each = c["d"] + 4 / c["block"] if c["kind"] == "decode8" else 2 * c["d"]
        return dict(bytes=c["B"] * (2 * c["Hkv"] * keys * each + c["Hq"] * c["Nq"] * (4 * c["d"] + 4)),
                    flops=4 * c["d"] * c["B"] * c["Hq"] * c["Nq"] * keys)
    N, w, S = c["N"], c["window"], c["sinks"]
    pairs = sum_pairs(N, w, S) * c["B"] * c["Hq"]
    q, kv = c["B"] * c["Hq"] * N * c["d"] * 2, c["B"] * c["Hkv"] * N * c["d"] * 2
    lse = c["B"] * c["Hq"] * N * 4
    if c["kind"] == "sink_fwd":
        return dict(bytes=2 * q + 2 * kv + lse, flops=4 * c["d"] * pairs)
    return dict(bytes=4 * q + 4 * kv + lse, flops=10 * c["d"] * pairs)


def sum_pairs(N, w, S):
    """Visible pairs of one head: each row's window, and the sinks behind it."""
    i = np.arange(N, dtype=np.int64)
    return int((np.minimum(i + 1, w) + np.minimum(np.maximum(i - w + 1, 0), S)).sum())


# ------------------------------------------------------------------ exact values
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode8": _exact_decode, "sink_decode": _exact_decode,
            "sink_fwd": _exact_sink, "sink_bwd": _exact_sink}[case["kind"]](s)


def _exact_append(s):
    c = s["case"]
    B, T, ps, bs, d = c["B"], c["tokens"], c["page"], c["block"], c["d"]
    L = s["seq_lens"].tolist()
    cu = s["cu_tokens"].tolist() if s["cu_tokens"] is not None else [i * (T // B) for i in range(B + 1)]
    table = s["block_table"].cpu().numpy()
    freq = s["inv_freq"].double()
    half = freq.numel()
    i = torch.arange(half, device=freq.device)
    ia, ib = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)

    def turned(x, pos):
        z = torch.polar(torch.ones(len(pos), 1, half, device=x.device, dtype=torch.float64), pos[:, None, None] * freq)
        x = x.double()
        y = x.clone()
        r = torch.complex(x[..., ia], x[..., ib]) * z
        y[..., ia], y[..., ib] = r.real, r.imag
        return y

    caches = {n: (s[n + "_cache"].double() if not bs else s[n + "_cache"].float()) for n in "kv"}
    scales = {n: s[n + "_scale"].clone() for n in "kv"} if bs else None
    qs = []
    for b in range(B):
        t0, t1 = cu[b], cu[b + 1]
        if t0 == t1:
            continue
        p0 = L[b] - (t1 - t0)
        pos = torch.arange(p0, L[b], device=freq.device).double()
        qs.append(turned(s["q"][t0:t1], pos))
        for n, x in (("k", turned(s["k"][t0:t1], pos)), ("v", s["v"][t0:t1].double())):
            step = bs or ps
            for lo in range(p0 // step * step, L[b], step):
                page, a, e = int(table[b, lo // ps]), max(lo, p0), min(lo + step, L[b])
                rows = x[a - p0:e - p0].transpose(0, 1)                       # [H, n, d]
                if not bs:
                    caches[n][page, :, a % ps:a % ps + e - a] = rows
                    continue
                sc, blk = scales[n][page, :, lo % ps // bs], slice(lo % ps, lo % ps + bs)
                amax = rows.abs().amax((1, 2))
                fresh = torch.exp2(torch.round(torch.log2((amax / 448).clamp_min(2.0 ** -40))) + 1)
                for _ in range(2):      # the smallest power of two that holds them, from one above it
                    fresh = torch.where((amax <= 224 * fresh) & (fresh > 2.0 ** -40), fresh / 2, fresh)
                if a > lo:
                    new = torch.where(amax <= 448.0 * sc.double(), sc.double(), fresh)
                    older = caches[n][page, :, blk][:, :a - lo] * (sc.double() / new)[:, None, None].float()
                    caches[n][page, :, blk][:, :a - lo] = older.to(E4M3).float()
                else:
                    new = fresh
                scales[n][page, :, lo % ps // bs] = new.float()
                caches[n][page, :, a % ps:a % ps + e - a] = (rows / new[:, None, None]).float().to(E4M3).float()
    q = torch.cat(qs) if qs else s["q"].double()
    if s["cu_tokens"] is None:
        q = q.view(B, T // B, c["Hq"], d).transpose(1, 2)
    out = dict(q=q, k_cache=caches["k"].double(), v_cache=caches["v"].double())
    if bs:
        out.update(k_scale=scales["k"].double(), v_scale=scales["v"].double())
    return out


def _exact_decode(s):
    c = s["case"]
    B, Hkv, Nq, d, ps = c["B"], c["Hkv"], c["Nq"], c["d"], c["page"]
    outs, lses = [], []
    for b, L in enumerate(s["seq_lens"].tolist()):
        j = torch.arange(L, device=s["q"].device)
        if c["window"]:
            j = j[(j > L - Nq - c["window"]) | (j < c["sinks"])]
        page, slot = s["block_table"][b].long()[j // ps], j % ps
        k, v = s["k_cache"][page, :, slot].double(), s["v_cache"][page, :, slot].double()
        if c["kind"] == "decode8":
            k = k * s["k_scale"][page, :, slot // c["block"]].double()[..., None]
            v = v * s["v_scale"][page, :, slot // c["block"]].double()[..., None]
        q = s["q"][b].double().view(Hkv, -1, Nq, d)
        S = torch.einsum("hgtd,jhd->hgtj", q, k) / d ** 0.5
        at = torch.arange(L - Nq, L, device=j.device)[:, None]
        hidden = j > at
        if c["window"]:
            hidden |= (j <= at - c["window"]) & (j >= c["sinks"])
        S[..., hidden] = -math.inf
        lse = torch.logsumexp(S, -1)
        outs.append(torch.einsum("hgtj,jhd->hgtd", (S - lse[..., None]).exp(), v).reshape(-1, Nq, d))
        lses.append(lse.reshape(-1, Nq))
    return torch.stack(outs), torch.stack(lses)


def _exact_sink(s):
    c = s["case"]
    N, d, w, group = c["N"], c["d"], c["window"], c["Hq"] // c["Hkv"]
    i = torch.arange(N, device=s["q"].device)
    gap = i[:, None] - i
    hidden = (gap < 0) | ((gap >= w) & (i >= c["sinks"]))
    got = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=i.device) for n in ("q", "k", "v")}
    lses = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device=i.device)
    for b in range(c["B"]):
        for h in range(c["Hq"]):
            q, k, v = s["q"][b, h].double(), s["k"][b, h // group].double(), s["v"][b, h // group].double()
            P = (q @ k.T).mul_(d ** -0.5).masked_fill_(hidden, -math.inf)
            lses[b, h] = torch.logsumexp(P, -1)
            if c["kind"] == "sink_fwd":
                got["q"][b, h] = P.sub_(lses[b, h][:, None]).exp_() @ v
                continue
            P.sub_(s["lse"][b, h].double()[:, None]).exp_()
            do = s["dout"][b, h].double()
            got["v"][b, h // group] += P.T @ do
            P *= (do @ v.T).sub_((do * s["out"][b, h].double()).sum(-1, keepdim=True))
            P *= d ** -0.5
            got["q"][b, h] = P @ k
            got["k"][b, h // group] += P.T @ q
    if c["kind"] == "sink_fwd":
        return got["q"], lses
    return got["q"], got["k"], got["v"]
