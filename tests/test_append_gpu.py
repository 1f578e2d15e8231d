"""Paged-cache append through the public binding against the fp64 reference.

Bounds: a rotated value carries the fp32 rotation's error, at most 4 roundings of
(|a| + |b|) 2^-24 plus an angle off by 2^-22 (|a| + |b|) at most: 2^-21 (|a| + |b|) in all.
bf16 adds half a step, 2^-8 relative (the type's eps / 2 of the value, counted up); E4M3 adds
half a step: 2^-4 relative, or 2^-10 of the scale below its normal range."""
import numpy as np
import pytest
import torch

from oracle import kv_append_fp64 as R

pytestmark = pytest.mark.gpu


def make(B, Hq, Hkv, d, page, block, counts, starts, seed, rot=None, theta=10000.0, boost=1.0, extra=3, tail=0):
    rs = np.random.RandomState(seed)
    counts, starts = np.asarray(counts), np.asarray(starts)
    lens = starts + counts
    width = max(1, int(-(-lens.max() // page)))
    need = [list(range(s // page, -(-(s + n) // page))) if n else [] for s, n in zip(starts, counts)]
    pool = sum(map(len, need)) + extra
    perm, table, at = rs.permutation(pool), np.full((B, width), -1, np.int32), 0
    for b, pages in enumerate(need):
        for lp in pages:
            table[b, lp] = perm[at]
            at += 1
    T = int(counts.sum()) + tail
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g).mul(boost).bfloat16().cuda()
    s = dict(q=qkv[:, :Hq * d].view(T, Hq, d), k=qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d),
             v=qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d), block_table=torch.from_numpy(table).cuda(),
             seq_lens=torch.from_numpy(lens.astype(np.int32)).cuda(),
             cu=torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda(), scales=None)
    rot = d if rot is None else rot
    s["inv_freq"] = (theta ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))).float().cuda() \
        if rot else None
    if block:
        codes = [torch.randn(pool, Hkv, page, d, generator=g).mul(60).to(torch.float8_e4m3fn).cuda() for _ in "kv"]
        s["caches"] = codes
        s["scales"] = [torch.exp2(torch.randint(-9, -3, (pool, Hkv, page // block), generator=g).float()).cuda()
                       for _ in "kv"]
    else:
        s["caches"] = [torch.randn(pool, Hkv, page, d, generator=g).bfloat16().cuda() for _ in "kv"]
    return s


def call(s, uniform=False, **kw):
    import exact_io_aware_72_b200 as attn
    sc = s["scales"] or (None, None)
    return attn.kv_append(s["k"], s["v"], s["caches"][0], s["caches"][1], s["block_table"], s["seq_lens"], q=s["q"],
                          cu_tokens=None if uniform else s["cu"], inv_freq=s["inv_freq"], k_scale=sc[0],
                          v_scale=sc[1], **kw)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(s, uniform=False, interleaved=False, positions=None):
    import exact_io_aware_72_b200 as attn
    attn.kv_append_debug_error()
    before = [c.view(torch.uint8).clone() if s["scales"] else c.clone() for c in s["caches"]]
    b_val = [f64(c) for c in s["caches"]]
    b_sc = [f64(c) for c in s["scales"]] if s["scales"] else [None, None]
    q = call(s, uniform, interleaved=interleaved, positions=positions)
    torch.cuda.synchronize()
    assert attn.kv_append_debug_error() == (0, 0)
    lens, cu = s["seq_lens"].cpu().numpy(), s["cu"].cpu().numpy()
    table = s["block_table"].cpu().numpy()
    rows = R.new_tokens(lens, cu)
    n = len(rows)
    pos = np.array([r[2] for r in rows]) if positions is None else positions.cpu().numpy()[:n]
    freq = f64(s["inv_freq"]) if s["inv_freq"] is not None else np.zeros(0)
    x = {k: f64(s[k][:n]) for k in "qkv"}
    turned = {k: R.rotate(x[k], pos, freq, interleaved) for k in "qk"}
    turned["v"] = x["v"]

    def slack(k):   # 2^-21 (|a| + |b|) at each element, zero where nothing turns
        a = np.abs(x[k])
        both = np.zeros_like(a)
        half = len(freq)
        i = np.arange(half)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        both[..., ia] = both[..., ib] = a[..., ia] + a[..., ib]
        return both * 2.0 ** -21

    got_q = f64(q)
    if uniform:
        got_q = got_q.transpose(0, 2, 1, 3).reshape(n, *got_q.shape[1:2], got_q.shape[3])
    err = np.abs(got_q[:n] - turned["q"])
    assert (err <= np.abs(turned["q"]) * 2.0 ** -8 + slack("q")).all()
    page = s["caches"][0].shape[2]
    written = np.zeros(s["caches"][0].shape[:3], bool)
    for t, b, p in rows:
        written[table[b][p // page], :, p % page] = True
    for name, cache, raw, val, sc, i in zip("kv", s["caches"], before, b_val, b_sc, (0, 1)):
        ref, ref_sc = R.append(turned[name], val, sc, table, lens, cu)
        lim = np.zeros(ref.shape)
        per = slack(name) if name == "k" else np.zeros_like(x["v"])
        for t, b, p in rows:
            lim[table[b][p // page], :, p % page] = per[t]
        got = f64(cache)
        if sc is None:
            assert (np.abs(got - ref) <= np.where(written[..., None], np.abs(ref) * 2.0 ** -8 + lim, 0)).all()
            continue
        got_sc = f64(s["scales"][i])
        assert np.array_equal(got_sc, ref_sc)     # random inputs: no maximum within 2^-21 of a power's edge
        block = page // sc.shape[2]
        s_at = np.repeat(ref_sc, block, 2)[..., None]
        bound = np.maximum(np.abs(ref) * 2.0 ** -4, 2.0 ** -10) + lim / s_at
        assert (np.abs(got - ref) <= np.where(written[..., None], bound, 0)).all()
    # bytes of slots that are neither new nor older rows of a rescaled block
    for cache, raw, sc, i in zip(s["caches"], before, b_sc, (0, 1)):
        now = cache.view(torch.uint8) if sc is not None else cache
        same = (now == raw).cpu().numpy().all(-1)
        keep = ~written
        if sc is not None:
            block = page // sc.shape[2]
            moved = np.repeat(f64(s["scales"][i]) != sc, block, 2)
            first_new = {(int(table[b][p // page]), p // block): p for t, b, p in reversed(rows)}
            held = np.zeros_like(written)
            for (phys, g), p in first_new.items():
                held[phys, :, p % page // block * block:p % page] = True
            keep &= ~(moved & held)
        assert same[keep].all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [0, 1, 16])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_one_token_each(cuda_ok, d, block, group):
    check(make(5, 2 * group, 2, d, 16, block, [1] * 5, [0, 15, 16, 1000, 131071], d + group), uniform=True)


@pytest.mark.parametrize("page,block", [(16, 0), (16, 16), (32, 4), (64, 64), (128, 32), (256, 256), (256, 0)])
def test_ragged_chunks(cuda_ok, page, block):
    check(make(7, 6, 2, 128, page, block, [1, 0, 300, 17, 64, 0, 129], [0, 5, 77, 16, 0, 40, 255], page + block))


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("Nq", [1, 2, 5, 16, 33])
def test_equal_sequences_take_the_decoding_layout(cuda_ok, block, Nq):
    check(make(4, 8, 4, 64, 16, block, [Nq] * 4, [0, 3, 15, 250], Nq, rot=32), uniform=True)


@pytest.mark.parametrize("rot", [0, 16, 64, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_part(cuda_ok, rot, interleaved):
    check(make(2, 4, 4, 128, 32, 0, [40, 3], [9, 0], rot, rot=rot), interleaved=interleaved)
    check(make(2, 4, 4, 128, 32, 32, [40, 3], [9, 0], rot, rot=rot), interleaved=interleaved)


def test_far_positions_and_given_positions(cuda_ok):
    s = make(2, 2, 2, 128, 64, 0, [5, 5], [(1 << 20) - 70, 12345678], 3, theta=500000.0)
    check(s)
    s = make(2, 2, 1, 64, 16, 16, [9, 4], [100, 200], 4)
    check(s, positions=torch.tensor([0, 7, 2 ** 31 - 1, -5, 3, 3, 3, 1 << 24, 9, 1, 2, 3, 4], dtype=torch.int32).cuda())


@pytest.mark.parametrize("boost", [2.0 ** -50, 0.01, 1000.0])
def test_blocks_that_held_tokens(cuda_ok, boost):
    # 2^-50: every scale at its floor or kept; 1000: every older block is rounded again
    check(make(6, 2, 3, 128, 64, 16, [1, 2, 30, 5, 16, 17], [1, 15, 33, 63, 8, 100], 5, boost=boost))
    check(make(3, 2, 3, 64, 32, 32, [1, 2, 70], [31, 5, 33], 6, boost=boost))


def test_many_sequences_and_rows_behind_the_last(cuda_ok):
    rs = np.random.RandomState(0)
    counts = rs.randint(0, 4, 100)
    s = make(100, 2, 2, 64, 16, 16, counts, rs.randint(0, 3000, 100), 7, tail=9)
    check(s)


def test_zero_rows_and_scale_floor(cuda_ok):
    import exact_io_aware_72_b200 as attn
    s = make(1, 1, 1, 64, 16, 16, [4], [0], 8)
    s["k"].zero_()
    s["v"].zero_()
    call(s)
    page = int(s["block_table"][0, 0])
    assert float(s["scales"][0][page, 0, 0]) == 2.0 ** -40 and float(s["caches"][0][page, 0, :4].float().abs().max()) == 0
    s["k"].fill_(1.0)
    s["seq_lens"] += 4
    attn.kv_append(s["k"], s["v"], *s["caches"], s["block_table"], s["seq_lens"], k_scale=s["scales"][0],
                   v_scale=s["scales"][1])
    got = s["caches"][0][page, 0, :8, 0].float() * s["scales"][0][page, 0, 0]
    assert got.tolist() == [0.0] * 4 + [1.0] * 4


def test_values_that_are_not_finite(cuda_ok):
    s = make(1, 1, 1, 64, 16, 16, [3], [0], 9, rot=0)
    s["v"].fill_(1.0)
    s["v"][0, 0, 0], s["v"][1, 0, 1], s["v"][2, 0, 2] = float("nan"), float("inf"), float("-inf")
    call(s)
    page = int(s["block_table"][0, 0])
    sc = float(s["scales"][1][page, 0, 0])
    row = s["caches"][1][page, 0, :3].float().cpu()
    assert sc == 2.0 ** -8 and torch.isnan(row[0, 0]) and row[1, 1] == 448 and row[2, 2] == -448
    assert int(torch.isnan(row).sum()) == 1


def test_no_tokens_and_no_queries(cuda_ok):
    import exact_io_aware_72_b200 as attn
    s = make(2, 2, 2, 64, 16, 0, [0, 0], [3, 4], 10)
    before = s["caches"][0].clone()
    assert call(s).shape == (0, 2, 64)
    assert torch.equal(before, s["caches"][0])
    s = make(2, 2, 2, 64, 16, 0, [2, 3], [3, 4], 10)
    assert attn.kv_append(s["k"], s["v"], *s["caches"], s["block_table"], s["seq_lens"], cu_tokens=s["cu"]) is None


def test_bad_sequences_and_pages_are_reported_and_skipped(cuda_ok):
    import exact_io_aware_72_b200 as attn
    for uniform in (False, True):
        s = make(3, 2, 2, 64, 16, 0, [2, 2, 2], [3, 40, 60], 11)
        lens = s["seq_lens"].clone()
        for bad in (1, 10 ** 6):        # fewer positions than new tokens; beyond the page table
            s["seq_lens"][1] = bad
            before = [c.clone() for c in s["caches"]]
            call(s, uniform)
            st, code = attn.kv_append_debug_error()
            assert st == 1 and code >> 20 == 1 and code & 0xFFFFF == 1
            p = int(s["block_table"][1, 2])
            assert torch.equal(before[0][p], s["caches"][0][p]) and torch.equal(before[1][p], s["caches"][1][p])
        s["seq_lens"].copy_(lens)
        p, s["block_table"][1, 2] = int(s["block_table"][1, 2]), 999
        before = [c.clone() for c in s["caches"]]
        call(s, uniform)
        st, code = attn.kv_append_debug_error()
        assert st == 1 and code >> 20 == 2 and code & 0xFFFFF == 1
        assert torch.equal(before[0][p], s["caches"][0][p])


def test_rows_of_bad_token_ranges_are_skipped(cuda_ok):
    import exact_io_aware_72_b200 as attn
    s = make(3, 2, 2, 64, 16, 0, [2, 2, 2], [3, 40, 60], 12)
    before = [c.clone() for c in s["caches"]]
    for cu in ([0, 2, 4, 99], [0, 4, 2, 6], [-1, 2, 4, 6]):
        s["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        call(s)
        assert attn.kv_append_debug_error()[0] == 1
    s["cu"].copy_(torch.tensor([0, 0, 0, 0], dtype=torch.int32))
    for c, b in zip(s["caches"], before):
        c.copy_(b)
    call(s)
    assert attn.kv_append_debug_error()[0] == 0 and torch.equal(before[0], s["caches"][0])


def test_captured_call_follows_the_lengths(cuda_ok):
    """A captured append, replayed with other lengths and tokens, equals eager calls."""
    s = make(3, 4, 2, 128, 16, 16, [1, 1, 1], [3, 14, 60], 13, extra=20)
    s["block_table"][:, :] = torch.arange(s["block_table"].numel(), dtype=torch.int32).view_as(s["block_table"]).cuda()
    twin = {k: ([c.clone() for c in v] if isinstance(v, list) else v.clone() if torch.is_tensor(v) else v)
            for k, v in s.items()}
    call(s, True)
    call(twin, True)
    out = torch.empty(3, 4, 1, 128, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        call(s, True, q_out=out)
    for i in range(3):
        for t in (s, twin):
            t["seq_lens"] += 1
            t["k"].copy_(torch.randn(t["k"].shape, generator=torch.Generator().manual_seed(i)).cuda() * (i + 1))
        s["q"].copy_(twin["q"])
        g.replay()
        want = call(twin, True)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for a, b in zip(s["caches"] + s["scales"], twin["caches"] + twin["scales"]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("page,block,d", [(32, 16, 128), (64, 4, 64), (256, 1, 128), (32, 16, 64), (128, 8, 128)])
def test_long_chunks_of_small_blocks(cuda_ok, page, block, d):
    """Enough tokens for runs of 32 slots a CTA: ragged starts and ends in either half of a run."""
    counts, starts = [2000, 1, 17, 0, 2900, 33], [5, 100, 15, 40, 0, 511]
    for boost in (1.0, 300.0):
        check(make(6, 3, 1, d, page, block, counts, starts, 21, boost=boost))
    check(make(6, 2, 2, d, page, block, counts, [s + 16 for s in starts], 22, rot=32), interleaved=True)


@pytest.mark.parametrize("block", [0, 16])
def test_batches_wider_than_a_cta(cuda_ok, block):
    """More sequences than threads of a CTA, some without new tokens, a bad one among them."""
    import exact_io_aware_72_b200 as attn
    rs = np.random.RandomState(23)
    counts, starts = rs.randint(0, 4, 700), rs.randint(0, 40, 700)
    counts[[255, 256, 511, 512]], counts[600:620] = [1, 3, 0, 2], 0
    check(make(700, 2, 1, 64, 16, block, counts, starts, 24, tail=5))
    counts[300] = 2
    s = make(700, 2, 1, 64, 16, block, counts, starts, 25)
    whole = [c.clone() for c in s["caches"]]
    s["seq_lens"][300] = 1                       # fewer positions than new tokens
    call(s)
    st, code = attn.kv_append_debug_error()
    assert st == 1 and code & 0xFFFFF == 300
    pages = lambda b: [int(s["block_table"][b, i]) for i in range(starts[b] // 16, -(-(starts[b] + counts[b]) // 16))]
    for c, w in zip(s["caches"], whole):
        same = (c.view(torch.uint8) == w.view(torch.uint8)).flatten(1).all(1).cpu().numpy()
        assert same[pages(300)].all()
        assert not any(same[pages(b)].any() for b in (299, 301, 699, 0) if counts[b])
