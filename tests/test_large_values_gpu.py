"""What the append writes, the 8-bit decoding step reads: values of any size up to 448 x 2^60 come
back, beside ordinary and tiny ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE, BLOCK = 8, 2, 128, 16, 16


def cached(v, splits, k=None):
    """Out of one query per head over the appended values v [T, HKV, D], all scores equal."""
    import exact_io_aware_72_b200 as attn
    T = v.shape[0]
    pages = -(-T // PAGE)
    codes = [torch.zeros(pages, HKV, PAGE, D, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.ones(pages, HKV, PAGE // BLOCK, device="cuda") for _ in "kv"]
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    attn.kv_append(torch.zeros_like(v) if k is None else k, v, *codes, table, lens, k_scale=scale[0], v_scale=scale[1])
    q = torch.ones(1, HQ, 1, D, dtype=torch.bfloat16, device="cuda")
    out, lse = attn.decode_kv8(q, *codes, *scale, table, lens, num_splits=splits)
    torch.cuda.synchronize()
    assert attn.kv_append_debug_error() == (0, 0) and attn.decode_kv8_debug_error() == (0, 0)
    value = codes[1].view(torch.float8_e4m3fn).double() * scale[1].double().repeat_interleave(BLOCK, 2)[..., None]
    value = value.transpose(1, 2).reshape(-1, HKV, D)[:T]
    return out.double()[0, :, 0], lse.double()[0, :, 0], value


@pytest.mark.parametrize("size", [1e-30, 1.0, 1e10, 1e15, 1e18, 5e20])
@pytest.mark.parametrize("splits", [1, 2])
def test_values_of_one_size(cuda_ok, size, splits):
    g = torch.Generator().manual_seed(1)
    T = 700
    v = (torch.randn(T, HKV, D, generator=g).clamp(-4, 4).double() * size / 4).bfloat16().cuda()
    out, lse, value = cached(v, splits)
    want = value.mean(0).repeat_interleave(HQ // HKV, 0)
    slack = value.abs().mean(0).repeat_interleave(HQ // HKV, 0)
    # equal weights: 2^-9 + 2^-11 of each value, the exponentials and their sum 2^-16; bf16 2^-8 of the result
    bound = want.abs() * 2.0 ** -8 + slack * (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -16) + 2.0 ** -133
    assert ((out - want).abs() <= bound).all(), ((out - want).abs() / bound).max()
    assert (lse - torch.tensor(float(T)).double().log()).abs().max() <= 2.0 ** -16


def test_one_block_of_large_values(cuda_ok):
    """A block of 1e20 among ordinary ones: where it weighs nothing, the others are what they were; where
    it is seen, it is all there is."""
    g = torch.Generator().manual_seed(2)
    T = 512
    v = torch.randn(T, HKV, D, generator=g).bfloat16().cuda()
    k = torch.zeros(T, HKV, D, dtype=torch.bfloat16, device="cuda")
    k[64:80] = -32.0             # scores lower by 32 x 128 / sqrt(128) = 362: no weight at all
    plain, _, _ = cached(v, 1, k)
    v[64:80] *= 1e20
    hidden, _, value = cached(v, 1, k)
    keep = [i for i in range(T) if not 64 <= i < 80]
    want = value[keep].mean(0).repeat_interleave(HQ // HKV, 0)
    slack = value[keep].abs().mean(0).repeat_interleave(HQ // HKV, 0)
    assert ((hidden - want).abs() <= want.abs() * 2.0 ** -8 + slack * (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -16)).all()
    assert torch.equal(hidden, plain)
    # the sum has every key, whatever their scales: zeros (scale 2^-40) beside the large ones
    z = v.clone()
    z[keep] = 0
    for splits in (1, 2):
        out, lse, value = cached(z, splits)
        want = value.mean(0).repeat_interleave(HQ // HKV, 0)
        slack = value.abs().mean(0).repeat_interleave(HQ // HKV, 0)
        assert ((out - want).abs() <= want.abs() * 2.0 ** -8 + slack * (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -16)).all()
        assert (lse - torch.tensor(float(T)).double().log()).abs().max() <= 2.0 ** -16
    seen, _, value = cached(v, 1)
    want = value.mean(0).repeat_interleave(HQ // HKV, 0)
    slack = value.abs().mean(0).repeat_interleave(HQ // HKV, 0)
    assert ((seen - want).abs() <= want.abs() * 2.0 ** -8 + slack * (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -16)).all()
