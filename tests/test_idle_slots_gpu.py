"""Idle slots of a padded batch (seq_lens 0) through both halves of a generation step: the append leaves
the cache alone, gives such a slot's queries as zeros and reports nothing; the decoding step gives
zeros.  The other slots get, bit for bit, what a batch without the idle ones gets."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HQ, HKV, WIDTH = 8, 2, 24


def state(B, n, d, block, lens, seed, page=64):
    g = torch.Generator().manual_seed(seed)
    pool = B * WIDTH
    s = dict(block_table=torch.randperm(pool, generator=g).int().view(B, WIDTH),
             seq_lens=torch.tensor(lens, dtype=torch.int32),
             qkv=torch.randn(B * n, (HQ + 2 * HKV) * d, generator=g).bfloat16(),
             inv_freq=(10000.0 ** (-torch.arange(d // 2) * 2 / d)).float())
    for c in "kv":
        x = torch.randn(pool, HKV, page, d, generator=g)
        s[c + "_cache"] = x.mul(60).to(torch.float8_e4m3fn) if block else x.bfloat16()
        s[c + "_scale"] = torch.exp2(torch.randint(-9, -4, (pool, HKV, page // block), generator=g).float()) if block else None
    return {k: v.cuda() if v is not None else None for k, v in s.items()}


def append(s, q_out=None):
    import exact_io_aware_72_b200 as attn
    d = s["k_cache"].shape[-1]
    T = s["qkv"].shape[0]
    q, k, v = (t.view(T, -1, d) for t in s["qkv"].split([HQ * d, HKV * d, HKV * d], 1))
    return attn.kv_append(k, v, s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], q=q, inv_freq=s["inv_freq"],
                          k_scale=s["k_scale"], v_scale=s["v_scale"], q_out=q_out)


def decode(s, q, splits, ws=None):
    import exact_io_aware_72_b200 as attn
    return attn.decode_kv8(q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["seq_lens"],
                           num_splits=splits, workspace=ws)


def only(s, live, n):
    """The same pool and tokens without the idle slots."""
    t = {k: v.clone() if v is not None else None for k, v in s.items()}
    t["block_table"], t["seq_lens"] = s["block_table"][live].contiguous(), s["seq_lens"][live].contiguous()
    t["qkv"] = s["qkv"].view(-1, n, s["qkv"].shape[1])[live].reshape(len(live) * n, -1).contiguous()
    return t


def raw(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("block", [0, 1, 16, 32, 64])
@pytest.mark.parametrize("n,d", [(1, 128), (2, 64), (33, 128), (200, 64)])
def test_append_passes_over_idle_slots(cuda_ok, block, n, d):
    import exact_io_aware_72_b200 as attn
    attn.kv_append_debug_error()
    lens = [0, 300, n, 0, 0, 1000, 0]
    s = state(len(lens), n, d, block, lens, n + d + block)
    live = [b for b, l in enumerate(lens) if l]
    idle = [b for b, l in enumerate(lens) if not l]
    t = only(s, live, n)
    s["block_table"][idle] = -1                     # not looked up
    s["qkv"].view(len(lens), n, -1)[idle] = float("nan")
    q_out = torch.full((len(lens), HQ, n, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = append(s, q_out)
    want = append(t)
    torch.cuda.synchronize()
    assert attn.kv_append_debug_error() == (0, 0)
    assert torch.equal(q[live], want) and not q[idle].any()
    for c in "kv":
        assert torch.equal(raw(s[c + "_cache"]), raw(t[c + "_cache"]))
        assert not block or torch.equal(s[c + "_scale"], t[c + "_scale"])


def test_every_slot_idle(cuda_ok):
    import exact_io_aware_72_b200 as attn
    attn.kv_append_debug_error()
    s = state(5, 1, 128, 16, [0] * 5, 1)
    before = {c: s[c].clone() for c in ("k_cache", "v_cache", "k_scale", "v_scale")}
    q = append(s)
    out, lse = decode(s, q, 2)
    torch.cuda.synchronize()
    assert attn.kv_append_debug_error() == (0, 0) and attn.decode_kv8_debug_error() == (0, 0)
    assert not q.any() and not out.any() and torch.isneginf(lse).all()
    assert all(torch.equal(raw(s[c]), raw(before[c])) for c in before)


def test_a_bad_length_beside_idle_slots_is_still_reported(cuda_ok):
    import exact_io_aware_72_b200 as attn
    attn.kv_append_debug_error()
    for bad in (1, -1, 10 ** 6):
        append(state(4, 2, 128, 16, [0, 300, bad, 0], 2))
        st, code = attn.kv_append_debug_error()
        assert st == 1 and code >> 20 == 1 and code & 0xFFFFF == 2


@pytest.mark.parametrize("splits", [1, 4])
def test_captured_padded_generation(cuda_ok, splits):
    """Slots fall idle and are taken again between replays of one captured step."""
    import exact_io_aware_72_b200 as attn
    attn.kv_append_debug_error()
    B, d = 4, 128
    s = state(B, 1, d, 16, [100, 0, 640, 1], 3)
    ws = attn.decode_kv8_workspace(B, HQ, HKV, 1, d, splits)
    step = lambda: decode(s, append(s), splits, ws)
    step()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out, lse = step()
    for i, lens in enumerate(([101, 0, 641, 2], [102, 1, 0, 3], [0, 2, 0, 4], [0, 0, 0, 5], [7, 3, 900, 0])):
        s["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        s["qkv"].copy_(torch.randn(s["qkv"].shape, generator=torch.Generator().manual_seed(i)))
        live = [b for b, l in enumerate(lens) if l]
        idle = [b for b, l in enumerate(lens) if not l]
        t = only(s, live, 1)
        graph.replay()
        want = decode(t, append(t), splits)
        torch.cuda.synchronize()
        assert attn.kv_append_debug_error() == (0, 0) and attn.decode_kv8_debug_error() == (0, 0)
        assert torch.equal(out[live], want[0]) and torch.equal(lse[live], want[1])
        assert not out[idle].any() and torch.isneginf(lse[idle]).all()
        assert all(torch.equal(raw(s[c]), raw(t[c])) for c in ("k_cache", "v_cache", "k_scale", "v_scale"))


def test_the_longest_length_may_be_an_idle_batchs(cuda_ok):
    """max_seq_len only picks the splits: a batch that has fallen idle passes 0, or what it has."""
    import exact_io_aware_72_b200 as attn
    s = state(3, 1, 128, 16, [0, 0, 0], 6)
    q = append(s)
    for longest in (0, 1, None):
        out, lse = attn.decode_kv8(q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                                   s["seq_lens"], max_seq_len=longest)
        assert not out.any() and torch.isneginf(lse).all()
    # more new tokens a slot than its table has positions
    q = torch.randn(2, HQ, 80, 128).bfloat16().cuda()
    out, lse = attn.decode_kv8(q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"][:2, :1].contiguous(),
                               s["seq_lens"][:2].contiguous(), max_seq_len=0)
    torch.cuda.synchronize()
    assert not out.any() and attn.decode_kv8_debug_error() == (0, 0)
