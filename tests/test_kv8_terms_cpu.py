"""The 8-bit terms of the decoding step's products, modelled on the host number for number: what the
header says of their rounding."""
import numpy as np


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
