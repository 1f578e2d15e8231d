"""The splits that a call chooses by itself, without a GPU: any longest length a padded batch can have."""
import pytest
import torch

from exact_io_aware_72_b200 import attn as A
from exact_io_aware_72_b200 import build as BLD


@pytest.mark.parametrize("longest,Nq,pages", [(0, 1, 3), (1, 4, 3), (None, 80, 1), (0, 80, 1), (48, 1, 3), (None, 1, 3)])
def test_lengths_shorter_than_the_new_tokens(monkeypatch, longest, Nq, pages):
    BLD.build()
    lib, seen = A.load_library(), []

    class Recorder:
        def __getattr__(self, name):
            return getattr(lib, name)

        @staticmethod
        def attn_decode_kv8(*args):
            seen.append(args)
            return 0

    monkeypatch.setattr(A, "load_library", Recorder)
    for name in ("_check", "_codes"):
        monkeypatch.setattr(A, name, lambda *a: None)
    monkeypatch.setattr(A, "_on_device", lambda index: A._NO_SWITCH)
    monkeypatch.setattr(A, "_stream_handle", lambda stream, index: 0)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    codes, scale = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.ones(3, 2, 1)
    A.decode_kv8(torch.zeros(2, 4, Nq, 64, dtype=torch.bfloat16), codes, codes, scale, scale,
                 torch.zeros(2, pages, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), max_seq_len=longest)
    assert seen
