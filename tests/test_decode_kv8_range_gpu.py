"""How far down the 8-bit decoding step holds its weights.

The product with V takes w_j = p_j c_j (p the softmax weight, c the V block's scale) as three
E5M2 numbers, scaled so that a row's largest, M, lies in [2^12, 2^15]:
* rounding to fp16: 2^-11 relative, or 2^-25 absolute where subnormal;
* each E5M2 term keeps three significant bits of what is left, the last one rounded to nearest: off by
  2^-9 of the weight, or by half of E5M2's smallest step, 2^-17, where that is more.
So a weight is off by at most (2^-9 + 2^-11) w + (2^-17 + 2^-25) / 2^12 M, and an output, the weights
divided by the exact sum l, by those errors times |code| / l.  The queries and keys here make the
scores exact sums of a few powers of two; the exponentials and their sum (fp32, at most 2^16
terms in a fixed tree of 2^-24 roundings) carry 2^-17.  bf16 then rounds by 2^-8 of the value."""
import numpy as np
import pytest
import torch

from tests.test_decode_kv8_gpu import run, values

pytestmark = pytest.mark.gpu

D, PAGE = 128, 64


def state(rank, vcode, vscale, rows=1):
    """Keys j whose score is -rank[j] (base 2, scale 1), V rows of codes vcode[j], and V scales of
    each block of 16; the query is (1, 1, 0, ...) and a key (a, b, 0, ...) with a + b its score."""
    L = len(rank)
    pages = -(-L // PAGE)
    score = -np.asarray(rank, np.float64) * np.log(2)   # natural units, as the kernel multiplies by log2(e)
    k = torch.zeros(pages * PAGE, D)
    # the largest E4M3 numbers first: what is left after three terms is below 2^-9 of the score
    left = torch.from_numpy(score)
    for i in range(4):
        t = (left * 8).float().to(torch.float8_e4m3fn).float()
        k[:L, i] = t
        left = left - t.double() / 8
    v = torch.zeros(pages * PAGE, D)
    v[:L] = torch.from_numpy(np.asarray(vcode, np.float32))
    lay = lambda x: x.view(pages, 1, PAGE, D).to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.zeros(1, rows, 1, D)
    q[..., :4] = 1.0
    sc = torch.ones(pages * PAGE // 16)
    sc[:len(vscale)] = torch.as_tensor(vscale, dtype=torch.float32)
    s = dict(q=q.bfloat16(), k_cache=lay(k), v_cache=lay(v), k_scale=torch.full((pages, 1, PAGE // 16), 0.125),
             v_scale=sc.view(pages, 1, PAGE // 16), block_table=torch.arange(pages, dtype=torch.int32)[None],
             seq_lens=torch.tensor([L], dtype=torch.int32))
    return s


def check(s, **kw):
    out, lse = run(s, scale=1.0, **kw)
    L = int(s["seq_lens"])
    key = values(s["k_cache"], s["k_scale"]).reshape(-1, D)[:L]
    code = s["v_cache"].view(torch.float8_e4m3fn).double().numpy().reshape(-1, D)[:L]
    c = np.repeat(s["v_scale"].double().numpy().reshape(-1), 16)[:L]
    x = key @ s["q"][0, 0, 0].double().numpy()
    p = np.exp(x - x.max())
    l = p.sum()
    want = (p * c) @ code / l
    w = p * c
    err_w = w * (2.0 ** -9 + 2.0 ** -11) + w.max() * (2.0 ** -29 + 2.0 ** -37)
    bound = np.abs(want) * 2.0 ** -8 + err_w @ np.abs(code) / l + (w @ np.abs(code)) / l * 2.0 ** -17
    got = out[0, :, 0].double().cpu().numpy()
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= bound).all(), f"{(err / bound).max():.3f} of the bound, off by {(err / np.abs(want)).max():.4f}"
    return want


@pytest.mark.parametrize("rank", [18.0, 20.5, 23.0, 25.5, 27.0])
@pytest.mark.parametrize("splits", [1, 3])
def test_many_small_weights_under_one_large(cuda_ok, rank, splits):
    """One key takes nearly all the weight and adds nothing in half of the columns; 20000 others, 2^-18
    to 2^-27 of it, are all there is in those."""
    g = np.random.default_rng(int(rank * 2))
    L = 20000
    r = np.concatenate([[0.0], rank + 0.5 * g.random(L - 1)])
    v = g.choice([1.0, 1.25, 1.5, 2.0], size=(L, D))
    v[0, :D // 2] = 0.0
    check(state(r, v, []), num_splits=splits)


@pytest.mark.parametrize("gap", [8, 16, 20, 24, 26])
def test_blocks_of_small_values_beside_one_of_large(cuda_ok, gap):
    """Equal softmax weights; one block's V scale lies 2^gap above the others', whose values are
    all there is in the columns where that block holds zeros."""
    g = np.random.default_rng(gap)
    L = 1024
    v = g.choice([64.0, 96.0, 128.0, 448.0], size=(L, D)) * g.choice([1.0, 1.0, 1.0, -1.0], size=(L, D))
    v[160:176, :D // 2] = 0.0
    sc = 1 + 0.5 * g.random(L // 16)
    sc[10] = 2.0 ** gap
    check(state(np.zeros(L), v, sc))


def test_a_maximum_that_creeps_up(cuda_ok):
    """Scores rise by a little under the bound at which the running maximum moves, tile after tile, and by a
    little over it: weights far above those the first tile set, none of them lost or overflowing."""
    for step in (2.9, 3.1, 5.9, 6.1):
        L = 128 * 7
        r = np.repeat(np.arange(7)[::-1] * step, 128)
        g = np.random.default_rng(int(step * 10))
        check(state(r, g.choice([1.0, -1.5, 2.0], size=(L, D)), []), num_splits=1)
