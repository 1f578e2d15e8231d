"""The forward with keys far and values near: K tiles come from HBM while V tiles are in L2, so that a
work item's loads land out of their order.  Every call gives the first call's bits, and those are
the reference's."""
import numpy as np
import pytest
import torch

from tests.parity import to_np

pytestmark = pytest.mark.gpu


def inputs(B, Hq, Hkv, N, d, seed, copies):
    """One q and v, and several copies of k (calls take them in turn, behind a sweep through L2)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v = (torch.randn(B, h, N, d, generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    return q, [k.clone() for _ in range(copies)], v


@pytest.mark.parametrize("B,Hq,Hkv,N,d,kw", [
    (2, 32, 32, 512, 128, dict(mask="causal")),
    (2, 32, 32, 1024, 128, dict(mask="causal")),
    (2, 32, 32, 512, 128, dict(mask="full")),
    (2, 32, 8, 768, 128, dict(mask="causal")),
    (2, 32, 32, 900, 128, dict(mask="sliding_window", window=400, sinks=4)),
    (2, 32, 32, 512, 64, dict(mask="causal")),
])
def test_every_call_gives_the_same_bits(cuda_ok, B, Hq, Hkv, N, d, kw):
    from exact_io_aware_72_b200 import debug_error, fwd
    debug_error()
    q, ks, v = inputs(B, Hq, Hkv, N, d, N + d, 4)
    sweep = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")   # more than L2
    ref_out, ref_lse = fwd(q, ks[0], v, **kw)
    bad = torch.zeros((), dtype=torch.long, device="cuda")
    for i in range(400):
        sweep.fill_(i & 127)
        v.sum()                                                        # the values are in L2 again
        out, lse = fwd(q, ks[i % 4], v, **kw)
        bad += (out != ref_out).any().long() + (lse != ref_lse).any().long()
    assert int(bad) == 0
    assert debug_error()[0] == 0
    rows = np.unique(np.concatenate([[0, N - 1], np.random.RandomState(N).randint(0, N, 30)]))
    for b, h in ((0, 0), (B - 1, Hq - 1)):
        hk = h // (Hq // Hkv)
        x = [to_np(t).astype(np.float64) for t in (q[b, h], ks[0][b, hk], v[b, hk])]
        s = x[0][rows] @ x[1].T * d ** -0.5
        i, j = rows[:, None], np.arange(N)
        seen = np.ones_like(s, bool) if kw["mask"] == "full" else j <= i
        if kw["mask"] == "sliding_window":
            seen &= (j > i - kw["window"]) | (j < kw["sinks"])
        s = np.where(seen, s, -np.inf)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        want = p @ x[2] / p.sum(1, keepdims=True)
        assert np.abs(to_np(ref_out[b, h])[rows] - want).max() <= 1e-2
        assert np.abs(to_np(ref_lse[b, h])[rows] - (m[:, 0] + np.log(p.sum(1)))).max() <= 1e-3
