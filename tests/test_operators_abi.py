"""The paged append, the 8-bit decoding step and the sinks option without a GPU: what is
refused before anything is launched, host-only sizes, the binding's checks, and the fp64
references against plainer forms of the same mathematics."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from exact_io_aware_72_b200 import attn as A
from exact_io_aware_72_b200 import build as BLD
from oracle import attention_sink_fp64 as S
from oracle import kv_append_fp64 as KA


@pytest.fixture(scope="module")
def lib():
    BLD.build()
    return A.load_library()


def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("GPU present")


# Fake, never-dereferenced device addresses: far apart, 256-byte aligned.
(Q, K, V, O, L, KC, VC, KS, VS, BT, SL, CU, POS, FREQ, WS, DO, DQ, DK, DV) = (0x10000000000 * (i + 1) for i in range(19))
BF16 = dict(k_scale=None, v_scale=None, scale_block=0)
SINKS = lambda n: ctypes.byref(A.FwdOptions(0, 0, 0, None, 0, 0, 0, 0, n))


# ------------------------------------------------------------------ append
def call_append(lib, **kw):
    a = dict(q=Q, k=K, v=V, q_stride=1024, k_stride=256, v_stride=256, q_out=O, k_cache=KC, v_cache=VC, k_scale=KS,
             v_scale=VS, block_table=BT, seq_lens=SL, cu_tokens=CU, positions=POS, inv_freq=FREQ, B=2, T=10, Hq=8,
             Hkv=2, d=128, rot_dim=128, num_pages=64, page_size=64, max_pages_per_seq=8, scale_block=16)
    a.update(kw)
    return lib.attn_kv_append(ctypes.byref(A.KvAppendArgs(**a)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k_cache=None), 1), (dict(v_cache=None), 1),
    (dict(block_table=None), 1), (dict(seq_lens=None), 1), (dict(q_out=None), 1), (dict(q=None), 1),
    (dict(k_scale=None), 1), (dict(v_scale=None), 1), (dict(scale_block=0), 1), (dict(scale_block=-16), 1),
    (dict(scale_block=24), 1), (dict(scale_block=128), 1),
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(Hq=0), 1), (dict(num_pages=0), 1),
    (dict(max_pages_per_seq=0), 1), (dict(B=3, cu_tokens=None), 1),
    (dict(d=96), 2), (dict(d=256), 2), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2),
    (dict(rot_dim=136), 1), (dict(rot_dim=-16), 1), (dict(rot_dim=0), 1), (dict(inv_freq=None), 1),
    (dict(rot_dim=24), 2),
    (dict(k_stride=128), 1), (dict(v_stride=248), 1), (dict(q_stride=1016), 1), (dict(k_stride=(1 << 31) + 8), 1),
    (dict(k_stride=257), 3), (dict(v_stride=260), 3), (dict(q_stride=1028), 3),
    (dict(k=K + 8), 3), (dict(v=V + 2), 3), (dict(q=Q + 8), 3), (dict(q_out=O + 8), 3), (dict(k_cache=KC + 8), 3),
    (dict(v_cache=VC + 8), 3), (dict(k_scale=KS + 2), 3), (dict(v_scale=VS + 1), 3), (dict(block_table=BT + 2), 3),
    (dict(seq_lens=SL + 1), 3), (dict(cu_tokens=CU + 2), 3), (dict(positions=POS + 2), 3), (dict(inv_freq=FREQ + 2), 3),
    (dict(q_out=Q), 1), (dict(k_cache=K), 1), (dict(v_cache=KC), 1), (dict(k_scale=VS), 1), (dict(k_scale=KC + 64), 1),
    (dict(v_scale=FREQ), 1), (dict(k_cache=BT), 1), (dict(q_out=SL), 1), (dict(k_scale=POS), 1),
    (dict(T=1 << 31), 1), (dict(B=1 << 31), 1), (dict(num_pages=1 << 31), 1), (dict(max_pages_per_seq=1 << 30), 1),
    (dict(B=1 << 20, max_pages_per_seq=1 << 20), 1), (dict(Hq=1 << 21, q_stride=1 << 28), 1),
])
def test_append_invalid_arguments_rejected_before_launch(lib, kw, status):
    assert call_append(lib, **kw) == status


def test_append_null_block_is_refused(lib):
    assert lib.attn_kv_append(None, None) == 1


def test_append_valid_arguments_reach_the_device_check(lib):
    no_gpu()
    assert call_append(lib) == 4
    assert call_append(lib, **BF16) == 4
    assert call_append(lib, cu_tokens=None) == 4
    assert call_append(lib, q=None, q_out=None, Hq=0, q_stride=0) == 4
    assert call_append(lib, rot_dim=0, inv_freq=None) == 4
    assert call_append(lib, T=0, k=None, v=None, q=None, q_out=None, cu_tokens=None) == 4
    # K and V as views of one projection's rows; the last row ends where the buffer does
    assert call_append(lib, k_stride=1536, v_stride=1536, q_stride=1536, k=Q + 2048, v=Q + 2560) == 4


@pytest.mark.parametrize("name,struct", [("attn_fwd_options", A.FwdOptions), ("attn_kv_append_args", A.KvAppendArgs)])
def test_binding_structs_match_the_header(name, struct, tmp_path):
    """Every field of the ctypes structs lies where a C compiler puts the header's."""
    cc, cuda = shutil.which("gcc"), os.path.join(os.path.dirname(os.path.dirname(BLD.nvcc_path())), "include")
    if cc is None or not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("no C compiler or CUDA headers")
    lines = "".join(f'printf("%zu\\n", offsetof({name}, {f[0]}));' for f in struct._fields_)
    (tmp_path / "o.c").write_text('#include <stddef.h>\n#include <stdio.h>\n#include "attn.h"\nint main(void) {' + lines +
                                  f'printf("%zu\\n", sizeof({name})); return 0; }}')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-I" + os.path.join(root, "include"), "-I" + cuda, "-o", str(tmp_path / "o"),
                    str(tmp_path / "o.c")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "o")], capture_output=True, text=True).stdout.split()]
    assert got == [getattr(struct, f[0]).offset for f in struct._fields_] + [ctypes.sizeof(struct)]


# ------------------------------------------------------------------ 8-bit decoding
def call_kv8(lib, q=Q, kc=KC, vc=VC, ks=KS, vs=VS, bt=BT, sl=SL, o=O, l=L, ws=WS, ws_bytes=None, B=2, Hq=8, Hkv=2,
             Nq=1, d=128, num_pages=64, page_size=16, max_pages=32, block=16, splits=4, scale=0.088, mask=1, window=0,
             sinks=0):
    if ws_bytes is None:
        ws_bytes = lib.attn_decode_kv8_workspace_bytes(B, Hq, Hkv, Nq, d, splits)
    return lib.attn_decode_kv8(q, kc, vc, ks, vs, bt, sl, o, l, ws, ws_bytes, B, Hq, Hkv, Nq, d, num_pages, page_size,
                               max_pages, block, splits, scale, mask, window, sinks, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(ks=None), 1), (dict(vs=None), 1),
    (dict(bt=None), 1), (dict(sl=None), 1), (dict(o=None), 1), (dict(l=None), 1), (dict(ws=None), 1),
    (dict(ws_bytes=16), 1), (dict(splits=1, ws=None), 1), (dict(splits=1, ws_bytes=128), 1),
    (dict(B=0), 1), (dict(Hq=6, Hkv=4), 1), (dict(Nq=0), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1),
    (dict(splits=0), 1), (dict(splits=1 << 20), 1), (dict(mask=3), 1), (dict(mask=-1), 1), (dict(mask=2, window=0), 1),
    (dict(sinks=-1), 1), (dict(sinks=4), 1), (dict(mask=0, sinks=4), 1), (dict(mask=2, window=64, sinks=-4), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(block=0), 1), (dict(block=-1), 1), (dict(block=12), 1), (dict(block=32), 1),
    (dict(d=96), 2), (dict(d=256), 2), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2),
    (dict(q=Q + 8), 3), (dict(kc=KC + 8), 3), (dict(vc=VC + 4), 3), (dict(o=O + 2), 3), (dict(l=L + 2), 3),
    (dict(ks=KS + 2), 3), (dict(vs=VS + 2), 3), (dict(bt=BT + 2), 3), (dict(sl=SL + 1), 3), (dict(ws=WS + 4), 3),
    (dict(o=Q), 1), (dict(l=KC + 64), 1), (dict(ws=BT), 1), (dict(o=SL), 1), (dict(l=O + 256), 1), (dict(ws=L), 1),
    (dict(o=KS), 1), (dict(ws=VS + 16), 1),
    (dict(num_pages=1 << 31), 1), (dict(max_pages=1 << 30), 1), (dict(B=1 << 20, Hq=1 << 20, Hkv=1 << 20), 1),
])
def test_decode_kv8_invalid_arguments_rejected_before_launch(lib, kw, status):
    if "B" in kw and kw["B"] > 1:
        kw = dict(kw, ws_bytes=1 << 60)
    assert call_kv8(lib, **kw) == status


def test_decode_kv8_valid_arguments_reach_the_device_check(lib):
    no_gpu()
    assert call_kv8(lib) == 4
    assert call_kv8(lib, splits=1) == 4
    assert call_kv8(lib, mask=0) == 4
    assert call_kv8(lib, mask=2, window=64, sinks=4) == 4
    assert call_kv8(lib, block=1) == 4


def test_decode_kv8_workspace_bytes(lib):
    rows, f = 2 * 8 * 3, lib.attn_decode_kv8_workspace_bytes
    assert f(2, 8, 2, 3, 128, 1) == 256
    assert f(2, 8, 2, 3, 128, 5) == 256 + -(-(rows * 5 * 4) // 256) * 256 + rows * 5 * 128 * 4
    for bad in ((0, 8, 2, 3, 128, 5), (2, 6, 4, 3, 128, 5), (2, 8, 2, 3, 96, 5), (2, 8, 2, 3, 128, 0),
                (2, 8, 2, 0, 128, 5), (1 << 20, 1 << 20, 1 << 20, 3, 128, 5)):
        assert f(*bad) == 0


def test_decode_kv8_num_splits_without_a_device(lib):
    no_gpu()
    f = lib.attn_decode_kv8_num_splits
    # 148 SMs of two CTAs assumed: one wave of items for one sequence or windows, else about
    # three waves of items of 16 to 48 tiles of 128 positions; never under four tiles for a split
    assert f(1, 64, 8, 1, 131072, 1, 0, 0) == 296 // 8
    assert f(32, 32, 32, 1, 131072, 1, 0, 0) == -(-(1024 + 1) // 48)
    assert f(1, 64, 8, 1, 1000, 1, 0, 0) == (8 + 1) // 4
    assert f(1, 32, 8, 1, 131072, 2, 4096, 0) == (32 + 1) // 4
    assert f(1, 32, 8, 1, 131072, 2, 4096, 256) == (32 + 1 + 2) // 4       # the sinks' two tiles
    assert f(8, 64, 8, 4, 32768, 1, 0, 0) == 3 * 296 // 64
    assert f(12, 16, 16, 1, 60000, 1, 0, 0) == -(-(469 + 1) // 48)
    assert f(30, 8, 8, 1, 8192, 1, 0, 0) == 3 * 296 // 240
    assert f(4, 32, 8, 1, 4096, 1, 0, 0) == (32 + 1) // 4
    assert f(1, 1, 1, 1, 1, 1, 0, 0) == 1
    for bad in ((1, 64, 8, 1, 0, 1, 0, 0), (1, 6, 4, 1, 100, 1, 0, 0), (1, 8, 8, 1, 100, 1, 0, 4),
                (1, 8, 8, 1, 100, 2, 0, 0), (1, 8, 8, 1, 100, 2, 8, -1), (1, 8, 8, 1, 100, 3, 0, 0)):
        assert f(*bad) == -1


# ------------------------------------------------------------------ sinks
def calls_with_sinks(lib, n, mask, window):
    """Statuses of the forward, the FP8 forward, the backward and the decoding step."""
    need = 1 << 40
    return [lib.attn_fwd_ex(Q, K, V, O, L, 1, 2, 2, 256, 64, 0.125, mask, window, None, SINKS(n)),
            lib.attn_fwd_fp8_ex(Q, K, V, 0.1, 0.1, 0.1, O, L, 1, 2, 2, 256, 128, 0.088, mask, window, None, SINKS(n)),
            lib.attn_bwd_ex(Q, K, V, O, L, DO, DQ, DK, DV, WS, need, 1, 2, 2, 256, 64, 0.125, mask, window, None,
                            SINKS(n)),
            lib.attn_decode_ex(Q, KC, VC, BT, SL, O, L, WS, need, 2, 8, 2, 1, 128, 64, 16, 32, 4, 0.088, mask, window,
                               None, SINKS(n))]


@pytest.mark.parametrize("n,mask,window", [(-1, 2, 16), (-1, 1, 0), (4, 0, 0), (4, 1, 0), (4, 2, 0), (4, 2, -1)])
def test_sinks_refused(lib, n, mask, window):
    assert calls_with_sinks(lib, n, mask, window) == [1] * 4


@pytest.mark.parametrize("n,window", [(4, 16), (0, 16), (256, 16), (1 << 40, 16), (4, 1 << 40), (1 << 40, 1 << 40)])
def test_sinks_reach_the_device_check(lib, n, window):
    no_gpu()
    assert calls_with_sinks(lib, n, 2, window)[:3] == [4] * 3


def test_backward_sink_workspace(lib):
    f, base = lib.attn_bwd_sink_workspace_bytes, lib.attn_bwd_workspace_bytes(1, 2, 4096)
    assert f(1, 2, 2, 4096, 64, 128, 0) == base                    # no sinks, or no keys out of sight
    assert f(1, 2, 2, 4096, 64, 4096, 4) == base
    need = f(1, 2, 2, 4096, 64, 128, 4)
    assert need > base
    for bad in ((0, 2, 2, 64, 64, 8, 4), (1, 2, 2, 64, 96, 8, 4), (1, 2, 2, 64, 64, 0, 4), (1, 2, 2, 64, 64, 8, -1),
                (1, 3, 2, 64, 64, 8, 4)):
        assert f(*bad) == 0
    need = f(1, 2, 2, 4096, 128, 128, 4)                           # d = 128: the dQ sums are used
    call = lambda ws, size: lib.attn_bwd_ex(Q, K, V, O, L, DO, DQ, DK, DV, ws, size, 1, 2, 2, 4096, 128, 0.088, 2, 128,
                                            None, SINKS(4))
    assert call(WS, need - 1) == 1
    assert call(WS + 8, need) == 3
    if not torch.cuda.is_available():
        assert call(WS, need) == 4


# ------------------------------------------------------------------ the binding
def test_bindings_validate_without_a_gpu():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    codes, sc = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.ones(3, 2, 1)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError):          # host tensors
        A.kv_append(x, x, cache, cache, table, lens)
    with pytest.raises(TypeError):
        A.kv_append(None, x, cache, cache, table, lens)
    with pytest.raises(ValueError):
        A.decode_kv8(torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16), codes, codes, sc, sc, table, lens)
    with pytest.raises(TypeError):
        A.decode_kv8(None, codes, codes, sc, sc, table, lens)
    with pytest.raises(ValueError):
        A.decode_kv8_num_splits(1, 8, 8, 1, 100, mask="banded")
    with pytest.raises(ValueError):
        A.decode_kv8_num_splits(1, 8, 8, 1, 100, mask="causal", sinks=4)
    with pytest.raises(ValueError):
        A.decode_kv8_workspace(1, 6, 4, 1, 64, 1, device="cpu")
    assert A.decode_kv8_workspace(1, 8, 4, 1, 64, 2, device="cpu").count_nonzero() == 0


# ------------------------------------------------------------------ the fp64 references
def test_reference_rounds_to_e4m3_as_the_type_does():
    x = np.concatenate([np.linspace(-460, 460, 4001), 2.0 ** np.linspace(-14, 8.7, 997), [0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = x.astype(np.float32)
    t = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(KA.e4m3(x), t)


def test_reference_scales_are_the_smallest_powers_of_two():
    amax = np.array([0.0, 1e-20, 448.0, np.nextafter(448.0, 500), 1.0, 7.0, 7.0000001, 3e38])
    s = KA.block_scale(amax)
    assert np.all(np.log2(s) == np.rint(np.log2(s))) and np.all(amax <= 448 * s)
    assert np.all((s == 2.0 ** -40) | (amax > 448 * s / 2))


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation_is_a_complex_product(interleaved):
    g = np.random.default_rng(3)
    x, pos, f = g.normal(size=(5, 3, 64)), np.array([0, 1, 7, 4096, 131071]), 10000.0 ** -(np.arange(16) / 16)
    y = KA.rotate(x, pos, f, interleaved)
    a, b = (np.arange(0, 32, 2), np.arange(1, 32, 2)) if interleaved else (np.arange(16), np.arange(16, 32))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[:, None] * f)[:, None]
    # fp64, angles to 131071: 2^-52 relative of each
    np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, rtol=0, atol=1e-10)
    assert np.array_equal(y[..., 32:], x[..., 32:])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (3, 2), (4, 9), (20, 3), (2, 50)])
def test_reference_forward_is_the_masked_softmax(window, sinks):
    g = np.random.default_rng(5)
    q, k, v = g.normal(size=(1, 4, 12, 8)), g.normal(size=(1, 2, 12, 8)), g.normal(size=(1, 2, 12, 8))
    out, lse, _ = S.forward(q, k, v, 0.3, window, sinks)
    x = torch.from_numpy(0.3 * np.einsum("bhid,bhjd->bhij", q, np.repeat(k, 2, 1)))
    i, j = torch.arange(12)[:, None], torch.arange(12)
    seen = (j <= i) & ((i - j < window) | (j < sinks))
    x = x.masked_fill(~seen, -torch.inf)
    np.testing.assert_allclose(lse, torch.logsumexp(x, -1).numpy(), rtol=0, atol=1e-13)
    want = torch.softmax(x, -1) @ torch.from_numpy(np.repeat(v, 2, 1))
    np.testing.assert_allclose(out, want.numpy(), rtol=0, atol=1e-13)


@pytest.mark.parametrize("window,sinks", [(1, 1), (3, 2), (20, 0)])
def test_reference_gradients_are_the_differences(window, sinks):
    g = np.random.default_rng(7)
    x = [g.normal(size=s) for s in ((1, 2, 9, 4), (1, 1, 9, 4), (1, 1, 9, 4))]
    dout, scale, step = g.normal(size=x[0].shape), 0.4, 1e-5
    got, _ = S.backward(*x, dout, scale, window, sinks)
    loss = lambda: (S.forward(*x, scale, window, sinks)[0] * dout).sum()
    for t, grad in zip(x, got):
        for at in [tuple(g.integers(n) for n in t.shape) for _ in range(12)]:
            keep = t[at]
            t[at] = keep + step
            up = loss()
            t[at] = keep - step
            down = loss()
            t[at] = keep
            # the second difference's step^2 term, and fp64 rounding over the step
            assert abs((up - down) / (2 * step) - grad[at]) < 1e-7 * (1 + abs(grad[at]))


def test_reference_decode_is_the_forwards_last_rows():
    g = np.random.default_rng(9)
    N, page, Nq = 23, 16, 3
    q, k, v = g.normal(size=(1, 4, N, 8)), g.normal(size=(1, 2, N, 8)), g.normal(size=(1, 2, N, 8))
    kc, vc = np.zeros((3, 2, page, 8)), np.zeros((3, 2, page, 8))
    table = np.array([[2, 0]])
    for j in range(N):
        kc[table[0, j // page], :, j % page], vc[table[0, j // page], :, j % page] = k[0, :, j], v[0, :, j]
    for window, sinks in ((4, 2), (1, 0), (9, 20)):
        want, want_lse, _ = S.forward(q, k, v, 0.25, window, sinks)
        out, lse, _, _ = S.decode(q[:, :, -Nq:], kc, vc, table, [N], 0.25, "sliding_window", window, sinks)
        np.testing.assert_allclose(out, want[:, :, -Nq:], rtol=0, atol=1e-14)
        np.testing.assert_allclose(lse, want_lse[:, :, -Nq:], rtol=0, atol=1e-14)
