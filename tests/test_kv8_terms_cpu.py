"""The 8-bit terms of the decoding step's products, modelled on the host number for number: what the
header says of their rounding."""
import os
import re

import numpy as np
import torch


def e5m2_terms(w):
    """A weight as the kernel splits it: fp16, its upper byte, the upper byte of what that leaves, and
    the rest rounded to an upper byte."""
    byte = np.uint16(0xff00)
    h = w.astype(np.float16)
    t1 = (h.view(np.uint16) & byte).view(np.float16)
    r = h - t1
    t2 = (r.view(np.uint16) & byte).view(np.float16)
    t3 = (((r - t2).view(np.uint16) + np.uint16(0x80)) & byte).view(np.float16)
    return [t.astype(np.float64) for t in (t1, t2, t3)]


def test_weights_keep_nine_bits_above_a_step():
    g = np.random.default_rng(1)
    top = 2.0 ** 12                      # where the running maximum sits, at the least
    for e in range(-30, 4):              # up to 2^15, where it must move
        w = (top * 2.0 ** (e - 1 + g.random(100000))).astype(np.float32).clip(max=2.0 ** 15)
        err = np.abs(sum(e5m2_terms(w)) - w.astype(np.float64))
        assert (err <= w * (2.0 ** -9 + 2.0 ** -11) + top * (2.0 ** -29 + 2.0 ** -37)).all()
        if e >= -19:
            assert (err <= w * (2.0 ** -9 + 2.0 ** -11)).all()
    # the largest weight and its terms are E5M2 numbers
    assert max(t.max() for t in e5m2_terms(np.float32([2.0 ** 15]))) <= 57344


def test_queries_are_two_e4m3_numbers():
    """Every bf16 element of a row whose largest has been scaled into [128, 256)."""
    x = torch.arange(1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[x < 256]
    first = x.to(torch.float8_e4m3fn).float()
    rest = (x - first - (x - first).to(torch.float8_e4m3fn).float()).abs().double()
    assert not rest[x >= 0.25].any()                      # 2^-9 of 128: exact from there on
    assert float(rest.max()) / 128 == 2.0 ** -17          # what the header gives, and no more
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "attn.h")
    assert re.search(r"two E4M3\s+\*?\s*terms \(exact to 2\^-17 of the row's largest element\)", open(header).read())
