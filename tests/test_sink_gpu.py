"""Sliding window with sinks: forward, backward and decoding through the public binding,
against the fp64 reference.

Forward bounds: weights in fp16 (2^-11 relative, and 2^-25 absolute below fp16's normal range
of a maximum that may lag; at most N of them), or bf16 (2^-8: spacing 2^-7,
biased truncation within 3/4 of it: 3 2^-9 counted up to 2^-7) or E4M3
(2^-4 of a weight); scores off by d + 8 fp32 roundings of the sum of |q k|; bf16 output 2^-8.
Backward bounds are the reference's (see there), and 2^-8 of the result."""
import numpy as np
import pytest
import torch

from harness.inputs import make_paged_kv, make_qkv, quantise_e4m3
from oracle import attention_sink_fp64 as R
from tests.parity import to_np

pytestmark = pytest.mark.gpu


def fwd_check(out, lse, ref, q, k, scale, weight):
    o, l, mean = ref
    N, d = q.shape[2:]
    g = q.shape[1] // k.shape[1]
    mass = scale * np.abs(q).sum(-1) * np.abs(k).max((2, 3)).repeat(g, 1)[..., None]
    slip = 2 * mass * (d + 8) * 2.0 ** -24 + 2.0 ** -18
    err = np.abs(to_np(out).astype(np.float64) - o)
    bound = np.abs(o) * 2.0 ** -8 + mean * (weight + slip[..., None]) + N * 2.0 ** -25 * 8
    assert np.isfinite(err).all() and (err <= bound).all(), (err / bound).max()
    gone = np.isneginf(l)
    got = to_np(lse).astype(np.float64)
    assert np.array_equal(gone, np.isneginf(got))
    assert (np.abs(got - np.where(gone, 0, l))[~gone] <= (slip + 2.0 ** -22 * np.abs(np.where(gone, 0, l)))[~gone]).all()


def forward(B, Hq, Hkv, N, d, window, sinks, seed, scale=None, sharp=False, **kw):
    from exact_io_aware_72_b200 import debug_error, fwd
    debug_error()
    q, k, v = make_qkv(B, Hq, Hkv, N, d, seed, sharp=sharp)
    scale = d ** -0.5 if scale is None else scale
    out, lse = fwd(q.cuda(), k.cuda(), v.cuda(), scale=scale, mask="sliding_window", window=window, sinks=sinks, **kw)
    assert debug_error()[0] == 0
    ref = R.forward(to_np(q), to_np(k), to_np(v), scale, window, sinks, kw.get("key_offset", 0))
    fwd_check(out, lse, ref, to_np(q).astype(np.float64), to_np(k).astype(np.float64), scale,
              2.0 ** -7 if kw.get("p_bf16") else 2.0 ** -11)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(2, 2), (4, 2), (3, 1), (8, 1)])
@pytest.mark.parametrize("N,window,sinks", [(1, 1, 1), (5, 2, 1), (300, 1, 4), (513, 100, 1), (700, 128, 128),
                                            (900, 130, 129), (1000, 5, 300), (640, 256, 127), (1300, 64, 640)])
def test_forward(cuda_ok, d, heads, N, window, sinks):
    forward(1, heads[0], heads[1], N, d, window, sinks, N + window)


def test_forward_batches_rescales_and_weights(cuda_ok):
    forward(2, 6, 3, 777, 128, 150, 9, 1, sharp=True)
    forward(2, 4, 4, 777, 64, 150, 200, 2, scale=1.0)
    forward(1, 4, 2, 900, 128, 150, 9, 3, p_bf16=True)
    forward(1, 4, 2, 900, 64, 150, 9, 4, p_bf16=True)
    for grid in (1, 3):
        forward(1, 4, 4, 900, 128, 150, 9, 5, grid_ctas=grid)


@pytest.mark.parametrize("off", [1, 100, 128, 500, 5000])
def test_forward_key_offset(cuda_ok, off):
    forward(1, 4, 2, 400, 128, 90, 5, off, key_offset=off)
    forward(1, 2, 2, 400, 64, 300, 200, off, key_offset=off)


def test_forward_fp8(cuda_ok):
    from exact_io_aware_72_b200 import fwd_fp8
    for N, window, sinks in ((700, 100, 3), (1000, 300, 140)):
        q, k, v = make_qkv(1, 4, 2, N, 128, 8, dtype=torch.float32)
        (q8, sq), (k8, sk), (v8, sv) = (quantise_e4m3(t) for t in (q, k, v))
        out, lse = fwd_fp8(q8.cuda(), k8.cuda(), v8.cuda(), sq, sk, sv, mask="sliding_window", window=window,
                           sinks=sinks)
        val = [t.view(torch.float8_e4m3fn).double().numpy() * s for t, s in ((q8, sq), (k8, sk), (v8, sv))]
        ref = R.forward(*val, 128 ** -0.5, window, sinks)
        fwd_check(out, lse, ref, val[0], val[1], 128 ** -0.5, 2.0 ** -4)


def test_forward_covering_masks_are_causal_bit_for_bit(cuda_ok):
    from exact_io_aware_72_b200 import fwd
    q, k, v = (t.cuda() for t in make_qkv(1, 4, 2, 600, 128, 9))
    ref = fwd(q, k, v, mask="causal")
    for window, sinks in ((600, 4), (500, 100), (1, 599), (1, 10 ** 9)):
        got = fwd(q, k, v, mask="sliding_window", window=window, sinks=sinks)
        assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    plain = fwd(q, k, v, mask="sliding_window", window=200)
    none = fwd(q, k, v, mask="sliding_window", window=200, sinks=0)
    assert torch.equal(plain[0], none[0]) and torch.equal(plain[1], none[1])


def backward(B, Hq, Hkv, N, d, window, sinks, seed, scale=None, **kw):
    from exact_io_aware_72_b200 import bwd, bwd_debug_error, fwd
    bwd_debug_error()
    q, k, v = make_qkv(B, Hq, Hkv, N, d, seed)
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(seed + 1)).bfloat16()
    g = [t.cuda() for t in (q, k, v)]
    out, lse = fwd(*g, scale=scale, mask="sliding_window", window=window, sinks=sinks)
    got = bwd(*g, out, lse, do.cuda(), scale=scale, mask="sliding_window", window=window, sinks=sinks, **kw)
    st, code = bwd_debug_error()
    assert st == 0, f"device error {code:#x}"
    ref, lim = R.backward(to_np(q), to_np(k), to_np(v), to_np(do), d ** -0.5 if scale is None else scale, window, sinks)
    for name, x, r, b in zip(("dq", "dk", "dv"), got, ref, lim):
        err = np.abs(to_np(x).astype(np.float64) - r)
        bound = np.abs(r) * 2.0 ** -8 + b + 1e-7
        assert np.isfinite(err).all() and (err <= bound).all(), (name, (err / bound).max())
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(2, 2), (4, 2), (3, 1)])
@pytest.mark.parametrize("N,window,sinks", [(5, 2, 1), (300, 1, 4), (513, 100, 1), (700, 128, 128), (900, 130, 129),
                                            (1000, 5, 300), (1300, 64, 640)])
def test_backward(cuda_ok, d, heads, N, window, sinks):
    backward(1, heads[0], heads[1], N, d, window, sinks, N + window)


def test_backward_deterministic_batches_and_few_ctas(cuda_ok):
    backward(2, 3, 3, 901, 128, 100, 7, 1, deterministic=True)
    backward(2, 4, 2, 901, 128, 100, 7, 2)
    for grid in (1, 5):
        backward(1, 2, 2, 901, 128, 100, 7, 3, grid_ctas=grid)
        backward(1, 4, 2, 901, 64, 100, 200, 4, grid_ctas=grid)


@pytest.mark.parametrize("kw", [dict(Hq=4, Hkv=2, d=128), dict(Hq=2, Hkv=2, d=128, deterministic=True),
                                dict(Hq=2, Hkv=1, d=64)])
def test_backward_repeats_bit_for_bit(cuda_ok, kw):
    a = backward(1, kw["Hq"], kw["Hkv"], 2000, kw["d"], 100, 5, 6, deterministic=kw.get("deterministic", False))
    b = backward(1, kw["Hq"], kw["Hkv"], 2000, kw["d"], 100, 5, 6, deterministic=kw.get("deterministic", False))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradient_against_differences(cuda_ok):
    """The reference's gradient against central differences of the reference's forward."""
    rs = np.random.RandomState(0)
    q, k, v, do = (rs.randn(1, h, 40, 64) for h in (2, 1, 1, 2))
    got, _ = R.backward(q, k, v, do, 0.125, 7, 3)
    for t, g in zip((q, k, v), got):
        for _ in range(6):
            at = tuple(rs.randint(0, n) for n in t.shape)
            old, h = t[at], 1e-5
            t[at] = old + h
            up = (R.forward(q, k, v, 0.125, 7, 3)[0] * do).sum()
            t[at] = old - h
            down = (R.forward(q, k, v, 0.125, 7, 3)[0] * do).sum()
            t[at] = old
            assert abs((up - down) / (2 * h) - g[at]) <= 1e-6 * max(1, abs(g[at]))


def step(B, Hq, Hkv, Nq, d, lens, page, window, sinks, seed, **kw):
    """A decoding step whose cache keeps only the pages the step may look up (others -1) and
    holds NaN in every slot no row sees."""
    from exact_io_aware_72_b200 import decode, decode_debug_error
    decode_debug_error()
    inp = make_paged_kv(B, Hq, Hkv, Nq, d, lens, page, seed, extra_pages=1)
    for b, L in enumerate(lens):
        for lp in range(-(-L // page)):
            phys = int(inp["block_table"][b, lp])
            pos = np.arange(lp * page, lp * page + page)
            seen = (pos < L) & ((pos > L - Nq - window) | (pos < sinks))
            for c in ("k_cache", "v_cache"):
                inp[c][phys][:, torch.from_numpy(~seen)] = float("nan")
            if not seen.any():
                inp["block_table"][b, lp] = -1
    g = {k: v.cuda() for k, v in inp.items()}
    out, lse = decode(g["q"], g["k_cache"], g["v_cache"], g["block_table"], g["seq_lens"], mask="sliding_window",
                      window=window, sinks=sinks, **kw)
    st, code = decode_debug_error()
    assert st == 0, f"device error {code:#x}"
    o, l, mean, mass = R.decode(to_np(inp["q"]), to_np(inp["k_cache"]), to_np(inp["v_cache"]),
                                inp["block_table"].numpy(), lens, None, "sliding_window", window, sinks)
    slip = 2 * mass * (d + 8) * 2.0 ** -24 + 2.0 ** -18
    err = np.abs(to_np(out).astype(np.float64) - o)
    # bf16 weights: half a step is 2^-8 (eps 2^-7), and so is the output's rounding
    bound = np.abs(o) * 2.0 ** -8 + mean * (2.0 ** -8 + slip[..., None])
    assert np.isfinite(err).all() and (err <= bound).all(), (err / bound).max()
    assert (np.abs(to_np(lse) - l) <= slip + 2.0 ** -22 * np.abs(l)).all()


@pytest.mark.parametrize("window", [1, 5, 127, 128, 300, 4096])
@pytest.mark.parametrize("sinks", [1, 4, 128, 200, 10 ** 9])
@pytest.mark.parametrize("Nq", [1, 3])
def test_decode(cuda_ok, window, sinks, Nq):
    lens = [Nq, 130, 1000, 2600]
    step(len(lens), 8, 2, Nq, 128, lens, 16, window, sinks, window + Nq)
    step(len(lens), 4, 4, Nq, 64, lens, 256, window, sinks, window + Nq, num_splits=3)


@pytest.mark.parametrize("rows", [40, 128, 150])
def test_decode_many_rows(cuda_ok, rows):
    step(2, rows, 1, 1, 128, [900, 2000], 64, 200, 70, rows, num_splits=2)
    step(2, rows // 2, 1, 2, 64, [900, 2000], 32, 200, 70, rows, grid_ctas=1)


def test_training_step_and_generation_agree(cuda_ok):
    """The forward's last rows equal a decoding step over a cache of the same keys, and the
    backward runs on them: the window with sinks means the same in all three."""
    from exact_io_aware_72_b200 import bwd, decode, fwd, kv_append
    B, Hq, Hkv, N, d, page, w, s = 2, 8, 2, 700, 128, 32, 150, 5
    q, k, v = (t.cuda() for t in make_qkv(B, Hq, Hkv, N, d, 11))
    out, lse = fwd(q, k, v, mask="sliding_window", window=w, sinks=s)
    pages = -(-N // page)
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(0)).int().view(B, pages).cuda()
    caches = [torch.zeros(B * pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    lens = torch.full((B,), N, dtype=torch.int32, device="cuda")
    rows = [t.transpose(1, 2).reshape(B * N, -1, d) for t in (q, k, v)]
    q2 = kv_append(rows[1], rows[2], *caches, table, lens, q=rows[0])
    assert torch.equal(q2, q)
    got, glse = decode(q[:, :, -4:].contiguous(), *caches, table, lens, mask="sliding_window", window=w, sinks=s)
    # two outputs, each within 2^-8 of its value and 2^-8 sum p|v| (|v| < 5 here) of the exact one
    assert (got.float() - out[:, :, -4:].float()).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -8) * 5
    assert (glse - lse[:, :, -4:]).abs().max() <= 1e-4
    grads = bwd(q, k, v, out, lse, torch.ones_like(q), mask="sliding_window", window=w, sinks=s)
    assert all(torch.isfinite(g.float()).all() for g in grads)


@pytest.mark.parametrize("N,window,sinks", [(1, 1, 1), (7, 6, 1), (300, 299, 1), (513, 10 ** 12, 4), (700, 10, 700), (260, 100, 200),
                                            (1030, 900, 140)])
def test_backward_of_covering_windows(cuda_ok, N, window, sinks):
    """The window and the sinks leave nothing out: causal gradients, from the sinks' own kernels or
    the fused one."""
    for heads, d in (((2, 2), 128), ((4, 2), 128), ((3, 1), 64)):
        backward(1, heads[0], heads[1], N, d, window, sinks, N)
