"""Calls with ``stream=`` and nothing of the caller's allocated beforehand, while the current stream is
busy: their workspaces are filled in that stream's order, and memory that the current stream still
uses, or takes next, is not theirs."""
import pytest
import torch

from tests.test_decode_kv8_gpu import make as make_kv8

pytestmark = pytest.mark.gpu

WINDOW = dict(mask="sliding_window", window=100, sinks=4)
BUSY = 40_000_000  # cycles: some 20 ms


def calls():
    import exact_io_aware_72_b200 as attn
    g = torch.Generator().manual_seed(12)
    s = {k: v.cuda() for k, v in make_kv8(3, 8, 2, 1, 128, [900, 40, 1500], 16, 16, 12).items()}
    bf = lambda c, sc: (c.view(torch.float8_e4m3fn).float() * sc.repeat_interleave(16, 2)[..., None]).bfloat16()
    pool = [bf(s["k_cache"], s["k_scale"]), bf(s["v_cache"], s["v_scale"])]
    q, k, v, do = (torch.randn(1, h, 700, 64, generator=g).bfloat16().cuda() for h in (4, 2, 2, 4))
    out, lse = attn.fwd(q, k, v, **WINDOW)
    codes = [torch.randn(1, 2, 300, 128, generator=g).to(torch.float8_e4m3fn).cuda() for _ in range(3)]
    new = torch.randn(2, 3, 2, 128, generator=g).bfloat16().cuda()
    qn = torch.randn(3, 8, 128, generator=g).bfloat16().cuda()
    return dict(
        decode_kv8=lambda **kw: attn.decode_kv8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                                s["block_table"], s["seq_lens"], num_splits=4, **kw),
        decode=lambda **kw: attn.decode(s["q"], *pool, s["block_table"], s["seq_lens"], num_splits=4, **kw),
        bwd=lambda **kw: attn.bwd(q, k, v, out, lse, do, **WINDOW, **kw),
        fwd=lambda **kw: attn.fwd(q, k, v, **WINDOW, **kw),
        fwd_fp8=lambda **kw: attn.fwd_fp8(*codes, 0.1, 0.1, 0.1, **kw),
        kv_append=lambda **kw: (attn.kv_append(new[0], new[1], *pool, s["block_table"], s["seq_lens"], q=qn, **kw),))


@pytest.mark.parametrize("name", ["decode_kv8", "decode", "bwd", "fwd", "fwd_fp8", "kv_append"])
def test_named_stream_beside_a_busy_current_stream(cuda_ok, name):
    call = calls()[name]
    want = call()
    torch.cuda.synchronize()
    sizes = [1 << n for n in range(9, 24)]
    side = torch.cuda.Stream()
    for late in (False, True):
        # Blocks of many sizes that the current stream is still to write ones into, and has given back.
        junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        for t in junk:
            t.fill_(0x3F)
        del junk
        if late:   # the call waits on its own stream while the current one goes on
            with torch.cuda.stream(side):
                torch.cuda._sleep(2 * BUSY)
        got = call(stream=side)
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x7F)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_dropped_outputs_wait_for_the_current_stream(cuda_ok):
    """An output that the current stream still reads is not handed to the named stream's next call."""
    call = calls()["fwd"]
    side = torch.cuda.Stream()
    want = call()[0]
    got = call(stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    copy = got.clone()
    del got
    others = []
    with torch.cuda.stream(side):
        for _ in range(4):
            others.append(torch.full_like(want, float("nan")))
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


@pytest.mark.parametrize("name", ["decode_kv8", "decode", "bwd", "kv_append"])
def test_named_stream_inside_a_capture(cuda_ok, name):
    """A call on a stream forked from the captured one: its buffers live in the graph's pool; one of its
    results is dropped while the capture goes on."""
    call = calls()[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    main, side, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        call(stream=side)
        got = call(stream=side)
        main.wait_stream(side)
        copies = [t.clone() for t in got]
    for _ in range(3):
        for t in (*got, *copies):
            t.fill_(1.0)
        graph.replay()
        junk = [torch.full((1 << 20,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(copies, want))
        del junk
