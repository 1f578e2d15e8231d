"""Decoding over an 8-bit paged cache through the public binding against the fp64 reference.

Bounds: the kernel's weights carry an error of at most 2^-9 (three E5M2 terms of 3 bits; both
the sum of weights and the output divide out only a common factor), so an output is off by at
most 2^-9 of sum_j p_j |v_j|; a query element of at most 2^-18 of its row's largest and
d fp32 roundings (2^-24 each) move a score by at most mass * (2^-18 * r + d 2^-23), with mass the
largest sum |q_i k_i| scale of the row and r the row's largest |q| over its typical one (16
covers normal rows); a score's error moves p by that relative amount, twice (numerator and sum).
bf16 then rounds by half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

from oracle import attention_sink_fp64 as R

pytestmark = pytest.mark.gpu


def make(B, Hq, Hkv, Nq, d, lens, page, block, seed, window=None, sinks=0, spread=0.5, extra=2, junk=True):
    rs = np.random.RandomState(seed)
    lens = np.asarray(lens)
    need = []
    for L in lens:
        keep = np.arange(L)
        if window is not None:
            keep = keep[(keep > L - Nq - window) | (keep < sinks)]
        need.append(sorted(set((keep // page).tolist())))
    pool = sum(map(len, need)) + extra
    perm, at = rs.permutation(pool), 0
    table = np.full((B, max(1, -(-int(lens.max()) // page))), -1, np.int32)
    used = np.zeros((pool, page), bool)
    for b, pages in enumerate(need):
        for lp in pages:
            table[b, lp] = perm[at]
            slots = np.arange(lp * page, lp * page + page)
            used[perm[at]] = slots < lens[b]
            if window is not None:
                used[perm[at]] &= (slots > lens[b] - Nq - window) | (slots < sinks)
            at += 1
    g = torch.Generator().manual_seed(seed)
    s = dict(q=torch.randn(B, Hq, Nq, d, generator=g).bfloat16(), block_table=torch.from_numpy(table),
             seq_lens=torch.from_numpy(lens.astype(np.int32)))
    for n in "kv":
        x = torch.randn(pool, Hkv, page, d, generator=g)
        sc = torch.exp2(torch.round(spread * 4 * torch.randn(pool, Hkv, page // block, generator=g)) - 7)
        if n == "k":
            sc = torch.full_like(sc, 2.0 ** -7) * (1 + torch.rand(sc.shape, generator=g))   # not powers of two
        codes = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        if junk:   # slots that the step does not see: NaN codes
            codes[torch.from_numpy(~used)[:, None, :, None].expand(codes.shape)] = 0x7F
        s[n + "_cache"], s[n + "_scale"] = codes, sc
    return s


def values(codes, scale):
    x = codes.view(torch.float8_e4m3fn).double().numpy()
    return x * np.repeat(scale.double().numpy(), codes.shape[2] // scale.shape[2], 2)[..., None]


def reference(s, mask="causal", window=None, sinks=0, scale=None):
    return R.decode(s["q"].double().numpy(), values(s["k_cache"], s["k_scale"]), values(s["v_cache"], s["v_scale"]),
                    s["block_table"].numpy(), s["seq_lens"].numpy(), scale, mask, window, sinks)


def run(s, **kw):
    import exact_io_aware_72_b200 as attn
    g = {k: v.cuda() for k, v in s.items()}
    out, lse = attn.decode_kv8(g["q"], g["k_cache"], g["v_cache"], g["k_scale"], g["v_scale"], g["block_table"],
                               g["seq_lens"], **kw)
    torch.cuda.synchronize()
    return out, lse


def compare(out, lse, ref, d):
    o, l, mean, mass = ref
    slip = 2 * mass * (2.0 ** -18 * 16 + d * 2.0 ** -23) + 2.0 ** -18   # the last: ex2 and log2 approximations
    err = np.abs(out.double().cpu().numpy() - o)
    bound = np.abs(o) * 2.0 ** -8 + mean * (2.0 ** -9 + slip[..., None]) + 1e-30
    assert np.isfinite(err).all()
    assert (err <= bound).all(), f"{(err / bound).max():.3f} of the bound"
    got = lse.double().cpu().numpy()
    idle = np.isneginf(l)
    assert np.array_equal(idle, np.isneginf(got))
    assert (np.abs(got - np.where(idle, 0, l))[~idle] <= (slip + 2.0 ** -22 * np.abs(np.where(idle, 0, l)))[~idle]).all()


def check(B, Hq, Hkv, Nq, d, lens, page, block, seed=0, mask="causal", window=None, sinks=0, scale=None, spread=0.5,
          **kw):
    import exact_io_aware_72_b200 as attn
    attn.decode_kv8_debug_error()
    s = make(B, Hq, Hkv, Nq, d, lens, page, block, seed, window if mask == "sliding_window" else None, sinks, spread)
    out, lse = run(s, mask=mask, window=window, sinks=sinks, scale=scale, **kw)
    st, code = attn.decode_kv8_debug_error()
    assert st == 0, f"device error {code:#x}"
    compare(out, lse, reference(s, mask, window, sinks, scale), d)


@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("d", [128, 64])
def test_single_token_ragged_batch(cuda_ok, d, group):
    lens = [1, 2, 127, 128, 129, 1000, 3000]
    check(len(lens), 2 * group, 2, 1, d, lens, 16, 16, d + group)


@pytest.mark.parametrize("page,block", [(16, 1), (16, 16), (32, 8), (64, 64), (128, 16), (256, 256), (256, 128)])
@pytest.mark.parametrize("splits", [1, 3, None])
@pytest.mark.parametrize("d", [64, 128])
def test_pages_blocks_and_splits(cuda_ok, page, block, splits, d):
    check(4, 8, 2, 1, d, [5, 300, 777, 2049], page, block, page + block, num_splits=splits)


@pytest.mark.parametrize("Nq,group", [(2, 8), (4, 8), (7, 8), (3, 1), (16, 8), (8, 16), (5, 30), (1, 32), (1, 64)])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_multi_token_steps(cuda_ok, Nq, group, splits, d):
    # rows per KV head 16, 32, 56, 3, 128 (two chunks), 128, 150, 32, 64
    check(4, group, 1, Nq, d, [Nq, Nq + 1, 200, 1500], 64, 16, Nq * 100 + group, num_splits=splits)


@pytest.mark.parametrize("mask", ["full", "causal"])
def test_masks_of_new_tokens(cuda_ok, mask):
    check(3, 6, 3, 5, 128, [5, 129, 640], 32, 32, 4, mask=mask)


@pytest.mark.parametrize("window", [1, 5, 127, 128, 300, 4096])
@pytest.mark.parametrize("sinks", [0, 1, 4, 128, 200])
@pytest.mark.parametrize("Nq", [1, 3])
def test_window_and_sinks(cuda_ok, window, sinks, Nq):
    lens = [Nq, 130, 1000, 2600]
    check(len(lens), 8, 2, Nq, 128, lens, 16, 16, window + sinks, mask="sliding_window", window=window, sinks=sinks)
    check(len(lens), 8, 2, Nq, 64, lens, 64, 4, window + sinks, mask="sliding_window", window=window, sinks=sinks,
          num_splits=2)


def test_window_that_covers_everything_is_causal(cuda_ok):
    s = make(2, 8, 2, 2, 128, [40, 700], 32, 32, 77)
    ref = run(s)
    for w in (700, 10 ** 9):
        for sinks in (0, 5, 10 ** 9):
            got = run(s, mask="sliding_window", window=w, sinks=sinks)
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("splits", [2, 7, 40])
def test_more_splits_than_tiles(cuda_ok, splits):
    check(3, 8, 2, 1, 128, [1, 300, 2000], 16, 16, splits, num_splits=splits)


@pytest.mark.parametrize("grid", [1, 3, 7])
def test_few_ctas_walk_many_items(cuda_ok, grid):
    check(6, 16, 4, 2, 128, [2, 129, 600, 2500, 33, 1024], 16, 16, grid, num_splits=3, grid_ctas=grid)
    check(6, 16, 4, 5, 64, [5, 129, 600, 2500, 33, 1024], 64, 64, grid, num_splits=2, grid_ctas=grid)


@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_scales_far_apart_and_large_scores(cuda_ok, spread):
    # V scales over 2^+-30 and scores that move the running maximum many times
    check(2, 8, 1, 2, 128, [900, 4000], 16, 16, 3, scale=0.6, spread=spread)
    check(2, 8, 8, 1, 64, [900, 4000], 32, 4, 4, scale=1.5, spread=spread, num_splits=5)


def test_rising_scores(cuda_ok):
    # every tile's scores lie above the one before: m moves at each tile
    s = make(1, 16, 1, 1, 128, [4096], 64, 64, 5, junk=False)
    codes = s["k_cache"].view(torch.float8_e4m3fn).float()
    for pos in range(4096):
        pg = int(s["block_table"][0, pos // 64])
        codes[pg, 0, pos % 64] = codes[pg, 0, pos % 64].abs() * (1 + pos // 128) / 32
    s["k_cache"] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    s["q"] = s["q"].abs()
    out, lse = run(s, num_splits=1, scale=1.0)
    compare(out, lse, reference(s, scale=1.0), 128)


def test_idle_slots_of_a_padded_batch(cuda_ok):
    import exact_io_aware_72_b200 as attn
    s = make(4, 8, 2, 2, 128, [300, 0, 2, 0], 16, 16, 6)
    for splits in (1, 3):
        out, lse = run(s, num_splits=splits)
        assert attn.decode_kv8_debug_error() == (0, 0)
        assert not out[[1, 3]].any() and torch.isneginf(lse[[1, 3]]).all()
        compare(out, lse, reference(s), 128)


def test_bad_lengths_and_pages_are_reported(cuda_ok):
    import exact_io_aware_72_b200 as attn
    s = make(3, 8, 2, 2, 128, [100, 50, 400], 16, 16, 7)
    ref = reference(s)
    for bad in (1, -1, 10 ** 6):
        s["seq_lens"][1] = bad
        for splits in (1, 3):
            out, lse = run(s, num_splits=splits)
            st, code = attn.decode_kv8_debug_error()
            assert st == 1 and code >> 20 == 1 and code & 0xFFFFF == 1
            assert not out[1].any() and torch.isneginf(lse[1]).all()
            compare(out[[0, 2]], lse[[0, 2]], [x[[0, 2]] for x in ref], 128)
    s["seq_lens"][1] = 50
    s["block_table"][2, 3] = 10 ** 6
    run(s)
    st, code = attn.decode_kv8_debug_error()
    assert st == 1 and code >> 20 == 2 and code & 0xFFFFF == 2


def test_nan_reaches_only_the_rows_that_see_it(cuda_ok):
    s = make(2, 8, 2, 1, 128, [200, 300], 16, 16, 8)
    s["k_cache"][int(s["block_table"][1, 3]), 1, 5, 7] = 0x7F
    out, _ = run(s)
    assert torch.isnan(out[1, 4:]).all() and torch.isfinite(out[1, :4].float()).all() and torch.isfinite(out[0].float()).all()
    s["q"][0, 2, 0, 3] = float("inf")
    out, _ = run(s)
    assert torch.isnan(out[0, 2]).all() and torch.isfinite(out[0, [0, 1, 3]].float()).all()


def test_repeatable_and_workspace_left_clean(cuda_ok):
    import exact_io_aware_72_b200 as attn
    s = {k: v.cuda() for k, v in make(5, 16, 2, 1, 128, [3000, 17, 900, 4000, 1], 16, 16, 9).items()}
    for splits, grid in ((1, 0), (4, 0), (4, 3)):
        ws = attn.decode_kv8_workspace(5, 16, 2, 1, 128, splits)
        first = None
        for _ in range(4):
            out = torch.full_like(s["q"], float("nan"))
            got = attn.decode_kv8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                                  s["seq_lens"], num_splits=splits, workspace=ws, grid_ctas=grid, out=out)
            torch.cuda.synchronize()
            assert int(ws[:64].view(torch.int32).abs().sum()) == 0     # the work counter
            first = first or [t.clone() for t in got]
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_one_workspace_for_steps_of_other_sizes_and_many_units(cuda_ok):
    """A workspace serves steps of other sizes one after another; 17000 sequences of one head."""
    import exact_io_aware_72_b200 as attn
    B = 17000
    ws = attn.decode_kv8_workspace(B, 1, 1, 1, 64, 2)
    for args, splits in (((3, 8, 2, 2, 128, [300, 2, 1000], 16, 16, 10), 4), ((B, 1, 1, 1, 64, [3] * B, 16, 16, 11), 2),
                         ((2, 64, 1, 2, 128, [900, 70], 32, 4, 12), 3), ((3, 8, 2, 2, 128, [300, 2, 1000], 16, 16, 10), 2)):
        s = make(*args)
        out, lse = run(s, num_splits=splits, workspace=ws)
        compare(out, lse, reference(s), args[4])
        assert int(ws[:64].view(torch.int32).abs().sum()) == 0


def test_append_and_decode_run_together(cuda_ok):
    """A prefill and single-token steps: appended codes, decoded, equal the reference on the cache's values."""
    import exact_io_aware_72_b200 as attn
    B, Hq, Hkv, d, page, block = 3, 8, 2, 128, 32, 16
    g = torch.Generator().manual_seed(1)
    width = 12
    table = torch.randperm(B * width, generator=g).int().view(B, width)
    s = dict(block_table=table.cuda(), k_scale=torch.ones(B * width, Hkv, page // block, device="cuda"),
             v_scale=torch.ones(B * width, Hkv, page // block, device="cuda"),
             k_cache=torch.full((B * width, Hkv, page, d), 0x7F, dtype=torch.uint8, device="cuda"),
             v_cache=torch.full((B * width, Hkv, page, d), 0x7F, dtype=torch.uint8, device="cuda"))
    inv_freq = (10000.0 ** (-torch.arange(d // 2) * 2 / d)).cuda()
    counts = [torch.tensor([100, 0, 33])] + [torch.ones(B, dtype=torch.long)] * 20
    lens = torch.zeros(B, dtype=torch.long)
    for n in counts:
        lens = lens + n
        T = int(n.sum())
        qkv = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g).mul(1 + 0.1 * int(lens[0] % 7)).bfloat16().cuda()
        cu = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]).int().cuda()
        s["seq_lens"] = lens.int().cuda()
        step = T == B
        q = attn.kv_append(qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d), qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d),
                           s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], q=qkv[:, :Hq * d].view(T, Hq, d),
                           cu_tokens=None if step else cu, inv_freq=inv_freq, k_scale=s["k_scale"],
                           v_scale=s["v_scale"])
    out, lse = attn.decode_kv8(q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                               s["seq_lens"])
    assert attn.kv_append_debug_error() == (0, 0) and attn.decode_kv8_debug_error() == (0, 0)
    host = {k: v.cpu() for k, v in s.items()}
    host["q"] = q.cpu()
    compare(out, lse, reference(host), d)
