"""The 8-bit decoding step's bounded waits: loaders that stop (at the host's word) leave every role
waiting; the waits run out, the roles leave together, the work counter goes back to zero, the host
reads ATTN_ERR_TIMEOUT, and the next step with the same workspace is right."""
import pytest
import torch

from tests.test_decode_kv8_gpu import compare, make, reference

pytestmark = pytest.mark.gpu

LIMIT = 20_000_000  # ns


def step(s, ws, **kw):
    import exact_io_aware_72_b200 as attn
    got = attn.decode_kv8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                          s["seq_lens"], workspace=ws, **kw)
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("group,d", [(8, 128), (8, 64), (32, 128), (32, 64)])   # 16- and 32-row products
@pytest.mark.parametrize("splits,grid", [(1, 0), (3, 0), (3, 2)])
@pytest.mark.parametrize("stall", [1, 2, 5, 12])    # before any load, in the first ring, in a later one
def test_loaders_that_stop(cuda_ok, group, d, splits, grid, stall):
    import exact_io_aware_72_b200 as attn
    B, Hkv, lens = 3, 2, [4000, 130, 5000]
    host = make(B, group * Hkv, Hkv, 1, d, lens, 64, 16, group + d)
    s = {k: v.cuda() for k, v in host.items()}
    ws = attn.decode_kv8_workspace(B, group * Hkv, Hkv, 1, d, splits)
    assert attn.decode_kv8_debug_error() == (0, 0)
    step(s, ws, num_splits=splits, grid_ctas=grid, inject_stall=stall, wait_timeout_ns=LIMIT)
    st, code = attn.decode_kv8_debug_error()
    assert st == attn.attn.ATTN_ERR_TIMEOUT and code != 0
    assert int(ws[:64].view(torch.int32).abs().sum()) == 0       # the work counter
    assert attn.decode_kv8_debug_error() == (0, 0)               # the word was cleared
    out, lse = step(s, ws, num_splits=splits, grid_ctas=grid)
    assert attn.decode_kv8_debug_error() == (0, 0)
    compare(out, lse, reference(host), d)


def test_a_stop_behind_the_last_tile_changes_nothing(cuda_ok):
    import exact_io_aware_72_b200 as attn
    host = make(2, 8, 2, 1, 128, [700, 128], 16, 16, 3)
    s = {k: v.cuda() for k, v in host.items()}
    ws = attn.decode_kv8_workspace(2, 8, 2, 1, 128, 1)
    out, lse = step(s, ws, num_splits=1, inject_stall=7, wait_timeout_ns=LIMIT)    # six tiles at most
    assert attn.decode_kv8_debug_error() == (0, 0)
    compare(out, lse, reference(host), 128)
