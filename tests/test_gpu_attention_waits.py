"""GPU tests of what the attention kernels do when a wait gives up: a barrier is
made to wait for an arrival that never comes.  The call ends, moe_read_status
reports the timeout, and the next call on the same workspace is right.  Nothing
faults or hangs: every wait is bounded, and a block lets its copies and
products land before it leaves."""
import os
import sys
import time

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_gpu_attention as base  # noqa: E402
from test_gpu_attention import BF, HF, gen_of, ints, rand, starts  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu

MOE_ERR_DEVICE_TIMEOUT = -6


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


def times_out(call, ws, wait, junk=False):
    """call() clean, with the wait held, and clean again on the same workspace."""
    set_wait = moe.lib().moe_debug_attn_wait_timeout
    want = call()
    assert moe.read_status(ws) == 0
    if junk:
        ws.fill_(0x81)
    assert set_wait(wait) == 0
    try:
        t0 = time.monotonic()
        call()
        torch.cuda.synchronize()
        # half a second for each of a block's roles, which may wait for one another, and for each of its copies, and
        # up to three rounds of blocks
        assert time.monotonic() - t0 < 10.0
        assert moe.read_status(ws) == MOE_ERR_DEVICE_TIMEOUT
    finally:
        assert set_wait(0) == 0
    assert torch.equal(call(), want)
    assert moe.read_status(ws) == 0


def test_setting_is_checked():
    set_wait = moe.lib().moe_debug_attn_wait_timeout
    assert set_wait(-1) == -1 and set_wait(99) == -1


@pytest.mark.parametrize("case", [
    ([5000, 3000], 0, 8, 2, 128, 16, BF),
    ([5000, 3000], 0, 8, 2, 64, 16, HF),
    ([4000] * 3, 0, 48, 2, 128, 64, BF),             # 24 heads share a key-value head
    ([9000, 40, 700], 1000, 8, 2, 128, 16, BF),      # beside a shared prefix
    ([40000, 30000], 0, 8, 2, 128, 64, BF),          # several slices per warp, and loads in flight
    ([40000, 30000], 300, 8, 2, 64, 64, HF),
], ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}-{sum(c[0])}-pre{c[1]}")
def test_decode_load(case):
    kv_lens, prefix, Hq, Hkv, D, page, dtype = case
    q, kc, vc, table, pre = base.decode_case(*case)
    B, n = len(kv_lens), ints(kv_lens)
    ws = moe.alloc_attn_workspace(B, B, Hq, Hkv, D)
    times_out(lambda: moe.attn_decode(q, kc, vc, table, n, pre, prefix, workspace=ws), ws, 1)


WAITS = ["keys", "stage", "query", "S", "P", "O", "half", "turn", "item", "next"]       # from 2 on


CASES = {
    # sequences, rows and keys of each, Hq, Hkv, D, page (0: packed), dtype
    "few": (2, 60, 900, 8, 2, 128, 0, BF),
    "many": (160, 50, 300, 4, 1, 128, 0, BF),    # more items than SMs: a block has asked for the next when it gives up
    "D64-paged": (160, 50, 900, 4, 1, 64, 16, HF),
}


@pytest.mark.parametrize("name,wait", [("few", w) for w in WAITS] + [("many", w) for w in ("stage", "P", "turn", "next")] +
                         [("D64-paged", w) for w in ("keys", "S", "O")])
def test_prefill_waits(name, wait):
    case = CASES[name]
    n, rows, keys, Hq, Hkv, D, page, dtype = case
    g = gen_of(7)
    q = rand(g, n * rows, Hq, D, dtype=dtype)
    q[..., 0] = 4
    qs = starts([rows] * n)
    ws = moe.alloc_attn_workspace(n * rows, n, Hq, Hkv, D)
    if page:
        per = (keys + page - 1) // page
        kc, vc = rand(g, per, Hkv, page, D, dtype=dtype), rand(g, per, Hkv, page, D, dtype=dtype)
        table = ints([list(range(per))] * n)     # the same pages for all
        kc[100 // page, :, 100 % page, 0] = 60   # in the second half of a block: a new scale
        lens = ints([keys] * n)

        def call():
            return moe.attn_prefill_paged(q, kc, vc, table, qs, lens, causal=False, workspace=ws)
    else:
        k, v = rand(g, n * keys, Hkv, D, dtype=dtype), rand(g, n * keys, Hkv, D, dtype=dtype)
        k[100::keys, :, 0] = 60
        ks = starts([keys] * n)

        def call():
            return moe.attn_prefill(q, k, v, qs, ks, causal=False, workspace=ws)
    # (where the answer about the next item never comes, nobody can tell whose word it leaves)
    times_out(call, ws, 2 + WAITS.index(wait), junk=wait != "next")


@pytest.mark.parametrize("wait", ["keys", "query", "P", "O"])
def test_shared_prefix_waits(wait):
    kv_lens, prefix, Hq, Hkv, D, page = [300, 40, 700], 5000, 8, 2, 128, 16
    q, kc, vc, table, pre = base.decode_case(kv_lens, prefix, Hq, Hkv, D, page, BF)
    n, B = ints(kv_lens), len(kv_lens)
    ws = moe.alloc_attn_workspace(B, B, Hq, Hkv, D)
    times_out(lambda: moe.attn_decode(q, kc, vc, table, n, pre, prefix, workspace=ws), ws, 2 + WAITS.index(wait))
