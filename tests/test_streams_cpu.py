"""What a call with ``stream=`` allocates itself belongs to that stream: its blocks come from the
stream's pool, are filled there, and go back there.  Shown without a GPU: the library is a
stand-in that launches nothing, the tensors are host tensors that pass for device ones, and every
allocation is recorded with the stream that was current when it was made."""
import contextlib
import types

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from exact_io_aware_72_b200 import attn as A

ALLOCATIONS = ("aten::empty", "aten::zeros", "aten::new_empty", "aten::empty_like", "aten::zeros_like", "aten::full")


class Streams(TorchDispatchMode):
    """Records (bytes, current stream) of each allocation, and the streams a tensor is recorded on."""

    def __init__(self):
        super().__init__()
        self.current, self.made, self.recorded = "current", [], []

    def __torch_dispatch__(self, func, types_, args=(), kwargs=None):
        t = func(*args, **(kwargs or {}))
        if func._schema.name in ALLOCATIONS:
            self.made.append((t, self.current))
        return t

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s.name
        yield
        self.current = before


class Library:
    """Every entry point succeeds without doing anything; sizes are given in bytes."""

    def __getattr__(self, name):
        return (lambda *a: 4096) if "workspace_bytes" in name else (lambda *a: 1 if "num_splits" in name else 0)


SIDE = types.SimpleNamespace(name="side", cuda_stream=1234, device_index=0, synchronize=lambda: None)


@pytest.fixture
def streams(monkeypatch):
    mode = Streams()
    monkeypatch.setattr(A, "load_library", Library)
    monkeypatch.setattr(A, "_check", lambda *a: None)
    monkeypatch.setattr(A, "_codes", lambda *a: None)
    monkeypatch.setattr(A, "_rows", lambda t, *a: t.stride(0))
    monkeypatch.setattr(A, "_on_device", lambda index: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(A, "_is_other", lambda s: s is not None and s.name != mode.current)
    monkeypatch.setattr(A, "_Current", mode.stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(name=mode.current))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: mode.recorded.append((t, s.name)))
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    return mode


def same(t, g):   # (a tensor may come back from the recorder as another object over its memory)
    return t.data_ptr() == g.data_ptr()


def inputs():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    by = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    q, kv, lse = bf(2, 4, 32, 64), bf(2, 2, 32, 64), torch.zeros(2, 4, 32)
    pool, codes, scale = bf(3, 2, 16, 64), by(3, 2, 16, 64), torch.ones(3, 2, 1)
    table, lens, new = i32(2, 1), i32(2), bf(2, 2, 64)
    window = dict(mask="sliding_window", window=8, sinks=2)
    return dict(
        fwd=lambda **k: A.fwd(q, kv, kv, **k),
        fwd_fp32=lambda **k: A.fwd(q, kv, kv, out_fp32=True, **k),
        fwd_fp8=lambda **k: A.fwd_fp8(by(2, 4, 32, 128), by(2, 2, 32, 128), by(2, 2, 32, 128), 1.0, 1.0, 1.0, **k),
        bwd=lambda **k: A.bwd(q, kv, kv, q, lse, q, **k),
        bwd_sinks=lambda **k: A.bwd(q, kv, kv, q, lse, q, **window, **k),
        decode=lambda **k: A.decode(q[:, :, :1].contiguous(), pool, pool, table, lens, num_splits=2, **k),
        decode_kv8=lambda **k: A.decode_kv8(q[:, :, :1].contiguous(), codes, codes, scale, scale, table, lens,
                                            num_splits=2, **k),
        kv_append=lambda **k: A.kv_append(new, new, pool, pool, table, lens, q=bf(2, 4, 64), **k))


@pytest.mark.parametrize("call", sorted(inputs()))
def test_a_named_stream_owns_what_its_call_allocates(streams, call):
    fn = inputs()[call]
    with streams:
        got = fn(stream=SIDE)
    got = got if isinstance(got, tuple) else (got,)
    own = [(t, s) for t, s in streams.made if t.dtype != torch.uint8 or call != "fwd_fp8"]  # (that call's inputs)
    own = [(t, s) for t, s in own if any(same(t, g) for g in got) or t.dtype == torch.float32 and t.dim() == 1]
    assert len(own) >= len(got) and all(s == "side" for _, s in own), [(tuple(t.shape), s) for t, s in own]
    # and what is handed to the caller is kept while the caller's current stream still uses it
    assert all(any(same(t, g) and s == "current" for t, s in streams.recorded) for g in got)


@pytest.mark.parametrize("name", [None, "current"])
@pytest.mark.parametrize("call", sorted(inputs()))
def test_on_the_current_stream_nothing_is_switched(streams, call, name, monkeypatch):
    monkeypatch.setattr(A, "_stream_handle", lambda stream, index: 0)
    fn = inputs()[call]
    with streams:
        fn(stream=name and types.SimpleNamespace(name=name, cuda_stream=0))
    assert streams.made and all(s == "current" for _, s in streams.made) and not streams.recorded


def test_host_calls_stage_on_the_named_stream(streams):
    host = torch.zeros(1, 2, 32, 64, dtype=torch.bfloat16)
    out, lse = torch.zeros_like(host), torch.zeros(1, 2, 32)
    monkey = pytest.MonkeyPatch()
    monkey.setattr(A, "_host_tensor", lambda t, *a: t)
    # the outputs are host tensors here, the staging buffers pass for device ones
    monkey.setattr(torch.Tensor, "is_cuda", property(lambda t: t is not out and t is not lse))
    try:
        with streams:
            A.fwd_host(host, host, host, out=out, lse=lse, device="cpu", stream=SIDE)
    finally:
        monkey.undo()
    assert len(streams.made) == 5 and all(s == "side" for _, s in streams.made)
