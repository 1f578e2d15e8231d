"""The append, the 8-bit decoding step and sinks as programs use them: captured and replayed,
on other streams, two at a time, on pools beyond 2^31 elements, and at the ends of the number
ranges."""
import numpy as np
import pytest
import torch

from oracle import attention_sink_fp64 as R

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, PAGE, BLOCK, WIDTH = 3, 8, 2, 128, 16, 16, 64


def cache_state(seed, lens):
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(B * WIDTH, generator=g).int().view(B, WIDTH)
    codes = lambda: torch.randn(B * WIDTH, HKV, PAGE, D, generator=g).mul(60).to(torch.float8_e4m3fn)
    scale = lambda: torch.exp2(torch.randint(-8, -4, (B * WIDTH, HKV, PAGE // BLOCK), generator=g).float())
    s = dict(k_cache=codes(), v_cache=codes(), k_scale=scale(), v_scale=scale(), block_table=table,
             seq_lens=torch.tensor(lens, dtype=torch.int32),
             qkv=torch.randn(B, (HQ + 2 * HKV) * D, generator=g).bfloat16())
    s = {k: v.cuda() for k, v in s.items()}
    s["inv_freq"] = (10000.0 ** (-torch.arange(D // 2) * 2 / D)).cuda()
    return s


def step(s, splits, ws, q_out=None, **kw):
    """One generation step: the new tokens into the cache, then the attention of their queries."""
    import exact_io_aware_72_b200 as attn
    q, k, v = s["qkv"].split([HQ * D, HKV * D, HKV * D], 1)
    q = attn.kv_append(k.view(B, HKV, D), v.view(B, HKV, D), s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                       q=q.view(B, HQ, D), inv_freq=s["inv_freq"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                       q_out=q_out)
    return attn.decode_kv8(q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["seq_lens"],
                           num_splits=splits, workspace=ws, **kw)


def capture(fn, stream):
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        got = fn()
    return g, got


@pytest.mark.parametrize("splits", [1, 5])
def test_captured_steps_equal_eager_ones(cuda_ok, splits):
    import exact_io_aware_72_b200 as attn
    lens = [100, 1, 700]
    a, b = cache_state(1, lens), cache_state(1, lens)
    ws = [attn.decode_kv8_workspace(B, HQ, HKV, 1, D, splits) for _ in range(2)]
    step(a, splits, ws[0])      # the library's first use of the device is outside the capture
    step(b, splits, ws[1])
    torch.cuda.synchronize()
    g, got = capture(lambda: step(a, splits, ws[0]), torch.cuda.Stream())
    for i in range(20):
        for s in (a, b):
            s["seq_lens"] += 1
            s["qkv"].copy_(torch.randn(s["qkv"].shape, generator=torch.Generator().manual_seed(i)))
        g.replay()
        want = step(b, splits, ws[1])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert torch.equal(a["k_cache"].view(torch.uint8), b["k_cache"].view(torch.uint8))
    assert attn.decode_kv8_debug_error() == (0, 0) and attn.kv_append_debug_error() == (0, 0)


def test_two_graphs_replayed_at_once(cuda_ok):
    """Two captured decoders with workspaces of their own, replayed on two streams at a time."""
    import exact_io_aware_72_b200 as attn
    splits, states, graphs = 6, [], []
    for i in range(2):
        s, stream = cache_state(2 + i, [900, 300 + 400 * i, 1000]), torch.cuda.Stream()
        ws = attn.decode_kv8_workspace(B, HQ, HKV, 1, D, splits)
        want = [t.clone() for t in step(s, splits, ws)]     # (the same tokens again: the same bytes)
        torch.cuda.synchronize()
        g, got = capture(lambda: step(s, splits, ws), stream)
        states.append((s, ws))
        graphs.append((g, stream, got, want))
    for _ in range(30):
        for g, stream, _, _ in graphs:
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for _, _, got, want in graphs:
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    for _, ws in states:
        assert int(ws[:64].view(torch.int32).abs().sum()) == 0


def test_another_stream_waits_for_its_own_work(cuda_ok):
    import exact_io_aware_72_b200 as attn
    s = cache_state(4, [500, 60, 1000])
    ws = attn.decode_kv8_workspace(B, HQ, HKV, 1, D, 4)
    want = step(s, 4, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    keep = s["qkv"].clone()
    s["qkv"].zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)        # the inputs appear late, on this stream
        s["qkv"].copy_(keep)
        got = step(s, 4, ws)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # a stream named in the call, while another one is current
    s["qkv"].zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        s["qkv"].copy_(keep)
    q, k, v = s["qkv"].split([HQ * D, HKV * D, HKV * D], 1)
    q = attn.kv_append(k.view(B, HKV, D), v.view(B, HKV, D), s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                       q=q.view(B, HQ, D), inv_freq=s["inv_freq"], k_scale=s["k_scale"], v_scale=s["v_scale"], stream=side)
    got = attn.decode_kv8(q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["seq_lens"],
                          num_splits=4, workspace=ws, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_captured_training_step_with_sinks(cuda_ok):
    """Forward and backward in one graph; grouped heads, so every sum has a fixed order."""
    import exact_io_aware_72_b200 as attn
    g = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(1, h, 1500, 64, generator=g).bfloat16().cuda() for h in (4, 2, 2, 4))

    def train():
        out, lse = attn.fwd(q, k, v, mask="sliding_window", window=200, sinks=4)
        return out, lse, *attn.bwd(q, k, v, out, lse, do, mask="sliding_window", window=200, sinks=4)
    train()
    torch.cuda.synchronize()
    graph, got = capture(train, torch.cuda.Stream())
    for i in range(3):
        for t in (q, k, v, do):
            t.copy_(torch.randn(t.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, train()))
    assert attn.bwd_debug_error()[0] == 0 and attn.debug_error()[0] == 0


@pytest.mark.parametrize("kind", ["bf16", "kv8", "kv8 blocks of 1"])
def test_pools_beyond_2_31_elements(cuda_ok, kind):
    """The last pages of a pool whose offsets need more than 32 bits give what a small pool gives."""
    import exact_io_aware_72_b200 as attn
    page, block, used = 128, 1 if kind.endswith("1") else 128, 12
    pool = (1 << 31) // (HKV * page * D) + 100
    g = torch.Generator().manual_seed(6)
    lens = torch.tensor([500, 130, 384], dtype=torch.int32).cuda()
    table = torch.randperm(used, generator=g).int().view(B, 4).cuda()
    counts = [300, 130, 1]
    T = sum(counts)
    cu = torch.tensor([0, 300, 430, 431], dtype=torch.int32).cuda()
    qkv = torch.randn(T, (HQ + 2 * HKV) * D, generator=g).bfloat16().cuda()
    q, k, v = (t.view(T, -1, D) for t in qkv.split([HQ * D, HKV * D, HKV * D], 1))
    q1 = torch.randn(B, HQ, 1, D, generator=g).bfloat16().cuda()
    dtype = torch.bfloat16 if kind == "bf16" else torch.uint8
    init = torch.randn(used, HKV, page, D, generator=g)
    init = init.bfloat16() if kind == "bf16" else init.mul(50).to(torch.float8_e4m3fn).view(torch.uint8)
    results = []
    for n in (used, pool):
        caches = [torch.zeros(n, HKV, page, D, dtype=dtype, device="cuda") for _ in "kv"]
        scales = [None, None] if kind == "bf16" else [torch.full((n, HKV, page // block), 2.0 ** -6, device="cuda")
                                                      for _ in "kv"]
        for c in caches:
            c[n - used:] = init.cuda()
        tab = table + (n - used)
        qr = attn.kv_append(k, v, *caches, tab, lens, q=q, cu_tokens=cu, k_scale=scales[0], v_scale=scales[1])
        if kind == "bf16":
            out = attn.decode(q1, *caches, tab, lens, mask="sliding_window", window=200, sinks=5)
        else:
            out = attn.decode_kv8(q1, *caches, *scales, tab, lens, mask="sliding_window", window=200, sinks=5)
        torch.cuda.synchronize()
        results.append([qr, *out] + [c[n - used:].clone() for c in caches] +
                       [s[n - used:].clone() for s in scales if s is not None])
        if n == pool:
            assert not any(bool(c[:n - used].any()) for c in caches)
        del caches, scales
    assert attn.kv_append_debug_error() == (0, 0) and attn.decode_kv8_debug_error() == (0, 0)
    assert all(torch.equal(x, y) for x, y in zip(*results))
    torch.cuda.empty_cache()


def test_scores_near_the_ends_of_fp32(cuda_ok):
    """One visible position: the output is its value whatever the score."""
    import exact_io_aware_72_b200 as attn
    v = torch.randn(1, 1, 16, 64).mul(50).to(torch.float8_e4m3fn).cuda()
    one = torch.ones(1, 1, 1, device="cuda")
    table, lens = torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.int32).cuda()
    for code in (448.0, -448.0):
        for qv in (2.0 ** -120, 1.0, 2.0 ** 60, 2.0 ** 105):
            k = torch.full((1, 1, 16, 64), code).to(torch.float8_e4m3fn).cuda()
            q = torch.full((1, 4, 1, 64), qv).bfloat16().cuda()
            out, lse = attn.decode_kv8(q, k, v, one, one, table, lens, scale=1.0)
            want = v[0, 0, 0].float()
            # the weight is off by 2^-9 at most in the product and not at all in the sum; bf16 by 2^-8
            assert ((out[0, :, 0].float() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -9)).all()
            score = 64 * code * qv
            # the score's and the logarithm's fp32 roundings
            assert ((lse.double() - score).abs() <= abs(score) * 2.0 ** -20 + 2.0 ** -18).all()


def test_small_probabilities_keep_their_gradients(cuda_ok):
    """One key takes nearly every row's weight; the others' gradients, some 1e-7 of it, stay as
    accurate as the large ones (their P is below fp16's normal range)."""
    import exact_io_aware_72_b200 as attn
    N, d, window = 300, 64, 40
    g = torch.Generator().manual_seed(8)
    for hq, hkv in ((2, 1), (2, 2)):
        q = 1 + 0.02 * torch.randn(1, hq, N, d, generator=g)
        k = 0.05 * torch.randn(1, hkv, N, d, generator=g)
        k[:, :, 0] = 1.0
        v, do = torch.randn(1, hkv, N, d, generator=g), torch.randn(1, hq, N, d, generator=g)
        q, k, v, do = (t.bfloat16() for t in (q, k, v, do))
        dev = [t.cuda() for t in (q, k, v)]
        out, lse = attn.fwd(*dev, scale=0.25, mask="sliding_window", window=window, sinks=1)
        got = attn.bwd(*dev, out, lse, do.cuda(), scale=0.25, mask="sliding_window", window=window, sinks=1)
        ref, lim = R.backward(*(t.double().numpy() for t in (q, k, v, do)), 0.25, window, 1)
        for name, x, r, b in zip(("dq", "dk", "dv"), got, ref, lim):
            err = np.abs(x.double().cpu().numpy() - r)
            bound = np.abs(r) * 2.0 ** -8 + b + 1e-30
            assert (err <= bound).all(), (name, (err / bound).max())
