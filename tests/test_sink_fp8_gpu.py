"""The FP8 forward with a sliding window and sinks against the fp64 reference, over head groupings,
lengths, windows and sink counts.

Bounds: products of codes are exact in fp32, scores take d + 8 fp32 roundings of the sum of |q k|; a
weight goes to the product with V as E4M3 of 2^8 p (p relative to a maximum that is a row's largest or
below it): off by 2^-4 of it, or by half of E4M3's smallest step, 2^-10 / 2^8 = 2^-18, where that is
more, for each of at most window + sinks keys; the sum that divides is of the unrounded p, at
least 1.  bf16 rounds by 2^-8 of the value."""
import numpy as np
import pytest
import torch

from harness.inputs import make_qkv_fp8
from oracle import attention_fp8 as O8
from oracle import attention_sink_fp64 as R
from tests.parity import to_np

pytestmark = pytest.mark.gpu


def check(B, Hq, Hkv, N, window, sinks, seed, scale=None, sharp=False, **kw):
    from exact_io_aware_72_b200 import debug_error, fwd_fp8
    debug_error()
    cpu = make_qkv_fp8(B, Hq, Hkv, N, 128, seed, device="cpu", sharp=sharp)
    (q8, sq), (k8, sk), (v8, sv) = cpu
    out, lse = fwd_fp8(q8.cuda(), k8.cuda(), v8.cuda(), sq, sk, sv, scale=scale, mask="sliding_window", window=window,
                       sinks=sinks, **kw)
    torch.cuda.synchronize()
    assert debug_error()[0] == 0
    q, k, v = (O8.dequantise(c.numpy(), s) for c, s in cpu)
    scale = 128 ** -0.5 if scale is None else scale
    o, l, mean = R.forward(q, k, v, scale, window, sinks)
    mass = scale * np.abs(q).sum(-1) * np.abs(k).max((2, 3)).repeat(Hq // Hkv, 1)[..., None]
    slip = 2 * mass * (128 + 8) * 2.0 ** -24 + 2.0 ** -18
    keys = min(N, window + sinks)
    bound = np.abs(o) * 2.0 ** -8 + mean * (2.0 ** -4 + slip[..., None]) + keys * 2.0 ** -18 * np.abs(v).max()
    err = np.abs(to_np(out).astype(np.float64) - o)
    assert np.isfinite(err).all() and (err <= bound).all(), (err / bound).max()
    assert (np.abs(to_np(lse).astype(np.float64) - l) <= slip + 2.0 ** -22 * np.abs(l)).all()
    # and, so that a lost tile cannot hide in the weights' 2^-4: the whole error is far below it
    assert np.linalg.norm(to_np(out) - o) <= 2.0 ** -4 * np.linalg.norm(o)


@pytest.mark.parametrize("heads", [(2, 2), (4, 2), (3, 1), (8, 1)])
@pytest.mark.parametrize("N,window,sinks", [(1, 1, 1), (5, 2, 1), (300, 1, 4), (513, 100, 1), (700, 128, 128),
                                            (900, 130, 129), (1000, 5, 300), (640, 256, 127), (1300, 64, 640)])
def test_shapes(cuda_ok, heads, N, window, sinks):
    check(1, heads[0], heads[1], N, window, sinks, N + window)


def test_batches_scales_and_few_ctas(cuda_ok):
    check(2, 6, 3, 777, 150, 9, 1, sharp=True)
    check(2, 4, 4, 777, 150, 200, 2, scale=0.5)
    for grid in (1, 3):
        check(1, 4, 4, 900, 150, 9, 5, grid_ctas=grid)


def test_covering_masks_are_causal_bit_for_bit(cuda_ok):
    from exact_io_aware_72_b200 import fwd_fp8
    args = [x for c, s in make_qkv_fp8(1, 4, 2, 600, 128, 9, device="cpu") for x in (c.cuda(), s)]
    args = args[0::2] + args[1::2]
    want = fwd_fp8(*args, mask="causal")
    for window, sinks in ((600, 4), (500, 100), (1, 599), (1, 10 ** 9)):
        got = fwd_fp8(*args, mask="sliding_window", window=window, sinks=sinks)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    plain = fwd_fp8(*args, mask="sliding_window", window=200)
    none = fwd_fp8(*args, mask="sliding_window", window=200, sinks=0)
    assert torch.equal(plain[0], none[0]) and torch.equal(plain[1], none[1])


def test_refusals(cuda_ok):
    import exact_io_aware_72_b200 as attn
    args = [x for c, s in make_qkv_fp8(1, 2, 2, 64, 128, 9, device="cpu") for x in (c.cuda(), s)]
    args = args[0::2] + args[1::2]
    for kw in (dict(mask="causal", sinks=4), dict(mask="full", sinks=4), dict(mask="sliding_window", window=8, sinks=-1)):
        with pytest.raises(attn.AttnError):
            attn.fwd_fp8(*args, **kw)
