"""What the backward with sinks takes as its workspace: the sums it uses, and no more (without a GPU)."""
import ctypes

import pytest
import torch

from exact_io_aware_72_b200 import attn as A
from exact_io_aware_72_b200 import build as BLD

# Fake, never-dereferenced device addresses: far apart, 256-byte aligned.
Q, K, V, O, L, DO, DQ, DK, DV, WS = (0x100000000000 * (i + 1) for i in range(10))
up = lambda n: -(-n // 256) * 256


@pytest.fixture(scope="module")
def lib():
    BLD.build()
    return A.load_library()


def parts_bytes(lib, B, Hq, Hkv, N, d, window, sinks):
    """The partial sums alone: dV and dK of every sink tile's rows, fp32, for each part."""
    f = lib.attn_bwd_sink_workspace_bytes
    n = f(B, Hq, Hkv, N, d, window, sinks) - f(B, Hq, Hkv, N, d, window, 0)
    unit = B * Hkv * -(-sinks // 128) * 2 * 128 * d * 4
    assert n % unit == 0 and n // unit > 1
    return n


def call(lib, size, B, Hq, Hkv, N, d, window, sinks, deterministic=0, ws=WS):
    opts = A.FwdOptions(0, 0, 0, None, 0, 0, 0, deterministic, sinks)
    return lib.attn_bwd_ex(Q, K, V, O, L, DO, DQ, DK, DV, ws, size, B, Hq, Hkv, N, d, 0.1, 2, window, None,
                           ctypes.byref(opts))


CASES = [(1, 32, 8, 16384, 128, 1024, 4, False), (1, 32, 8, 4099, 64, 300, 130, False), (2, 3, 1, 5001, 128, 500, 4, True),
         (1, 2, 2, 4096, 64, 128, 4, False), (1, 2, 2, 4096, 128, 128, 4, True), (1, 2, 2, 4096, 128, 128, 4, False)]


@pytest.mark.parametrize("case", CASES)
def test_the_sizes_used_are_the_sizes_needed(lib, case):
    B, Hq, Hkv, N, d, window, sinks, det = case
    fused = Hq == Hkv and d == 128 and not det
    parts = parts_bytes(lib, *case[:7])
    need = up(lib.attn_bwd_workspace_bytes(B, Hq, N) if fused else 4 * B * Hq * N) + parts
    size = lib.attn_bwd_sink_workspace_bytes(*case[:7])
    if Hq != Hkv:
        assert size == need                 # shared heads never sum dq in the workspace
    assert size >= need
    # (one byte less is refused as it stands; the exact size only fails for want of a GPU)
    assert call(lib, need - 1, *case[:7], deterministic=int(det)) == 1
    if not torch.cuda.is_available():
        assert call(lib, need, *case[:7], deterministic=int(det)) == 4
    assert call(lib, need, *case[:7], deterministic=int(det), ws=WS + 4) == 3


@pytest.mark.parametrize("case", CASES)
def test_the_binding_allocates_that_much(lib, case, monkeypatch):
    B, Hq, Hkv, N, d, window, sinks, det = case
    given = []

    class Recorder:
        def __getattr__(self, name):
            return getattr(lib, name)

        @staticmethod
        def attn_bwd_ex(*args):
            given.append(args[10])
            return 0

    monkeypatch.setattr(A, "load_library", Recorder)
    monkeypatch.setattr(A, "_check", lambda *a: None)
    monkeypatch.setattr(A, "_on_device", lambda index: A._NO_SWITCH)
    monkeypatch.setattr(A, "_stream_handle", lambda stream, index: 0)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    q, kv = torch.empty(B, Hq, N, d, dtype=torch.bfloat16), torch.empty(B, Hkv, N, d, dtype=torch.bfloat16)
    A.bwd(q, kv, kv, q, torch.empty(B, Hq, N), q, mask="sliding_window", window=window, sinks=sinks, deterministic=det)
    fused = Hq == Hkv and d == 128 and not det
    own = lib.attn_bwd_workspace_bytes(B, Hq, N) if fused else 4 * B * Hq * N
    assert given == [up(own) + parts_bytes(lib, *case[:7])]
