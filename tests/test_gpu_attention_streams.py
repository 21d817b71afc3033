"""GPU tests of attention calls on another stream than the caller's: what a call
allocates is neither memory that work queued on the caller's stream still uses,
nor given away while that stream uses the result."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_gpu_attention as base  # noqa: E402
from test_gpu_attention import BF, ints, packed_case, starts  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


def long_work():
    """Some milliseconds on the current stream."""
    a = torch.ones(4096, 4096, device="cuda")
    for _ in range(12):
        a = a @ a * 1e-4
    return a


def calls():
    lens, prefix, Hq, Hkv, D, page = [2000, 45, 800], 1000, 8, 2, 128, 16
    q, kc, vc, table, pre = base.decode_case(lens, prefix, Hq, Hkv, D, page, BF)
    rows, k, v = packed_case([300], [3000], Hq, Hkv, D, BF, 61)
    prompt = torch.cat([rows] * 2)
    qs, ks, n, ps = starts([300]), starts([3000]), ints(lens), ints([0, 500, 540, 600])
    rope = base.rope_case(200, Hq, Hkv, D, 128, False, True, 16, BF)
    return {
        "decode": (lambda **s: moe.attn_decode(q, kc, vc, table, n, pre, prefix, **s), (3, 3)),
        "prefill": (lambda **s: moe.attn_prefill(rows, k, v, qs, ks, **s), (300, 1)),
        "paged": (lambda **s: moe.attn_prefill_paged(prompt, kc, vc, table, ps, n, **s), (600, 3)),
        "rope": (lambda **s: moe.rope_append(*rope, **s), (200, 0)),
    }, (Hq, Hkv, D)


@pytest.mark.parametrize("name", ["decode", "prefill", "paged", "rope"])
def test_memory_in_use_on_the_callers_stream(name):
    """Blocks of the sizes that the call allocates are freed while work queued on
    the caller's stream still writes to them."""
    made, shape = calls()
    call, (T, n_seq) = made[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    freed = [torch.empty_like(want) for _ in range(3)]
    freed += [moe.alloc_attn_workspace(T, n_seq, *shape) for _ in range(3)]
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    long_work()
    for t in freed:
        t.fill_(63)
    del t, freed
    got = call(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("name", ["decode", "prefill", "paged", "rope"])
def test_result_in_use_on_the_callers_stream(name):
    """The result is freed while the caller's stream has yet to read it; the
    other stream's next allocations must not get its memory."""
    made, _ = calls()
    call, _ = made[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    long_work()
    copy = torch.empty_like(want)
    copy.copy_(got)
    del got
    with torch.cuda.stream(side):
        others = [torch.empty_like(want).fill_(63) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
    del others
