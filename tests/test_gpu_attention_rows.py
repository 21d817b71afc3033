"""GPU tests of rows that belong to no sequence: q_starts that begin after 0 or
end before T are reported, and the rows outside are left as they were."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_reference as ref  # noqa: E402
import test_gpu_attention as base  # noqa: E402
from test_gpu_attention import BF, MOE_ERR_DEVICE, gen_of, ints, rand  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


@pytest.mark.parametrize("q_starts", [[0, 30, 33], [7, 40, 50], [4, 20, 41], [0, 0, 0], [0, 70, 50], [0, 30, -4]],
                         ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("keys", [90, 4000], ids=["whole", "split"])
@pytest.mark.parametrize("paged", [False, True], ids=["packed", "paged"])
def test_uncovered_rows(q_starts, keys, paged):
    T, Hq, Hkv, D, page = 50, 8, 2, 128, 16
    lens = [keys, 40]
    q = rand(gen_of(1), T, Hq, D, mul=2.5)
    ws = moe.alloc_attn_workspace(T, 2, Hq, Hkv, D)
    kc, vc, table, _ = base.page_pool(lens, page, Hkv, D, BF, 2)
    k, v = ([ref.paged(c, table[s, :(n + page - 1) // page], n) for s, n in enumerate(lens)] for c in (kc, vc))
    packed = [torch.cat(x, 1).transpose(0, 1).contiguous() for x in (k, v)]
    starts = ints([0, lens[0], sum(lens)])

    def call(qs):
        out = torch.full((T, Hq, D), 7.0, dtype=BF, device="cuda")
        lse = torch.full((T, Hq), 7.0, device="cuda")
        if paged:
            moe.attn_prefill_paged(q, kc, vc, table, ints(qs), ints(lens), causal=False, out=out, lse=lse, workspace=ws)
        else:
            moe.attn_prefill(q, *packed, ints(qs), starts, causal=False, out=out, lse=lse, workspace=ws)
        return out, lse, moe.read_status(ws)
    assert call([0, 20, T])[2] == 0                    # an earlier call's parts lie in the workspace
    out, lse, status = call(q_starts)
    assert status == MOE_ERR_DEVICE
    covered = torch.zeros(T, dtype=torch.bool, device="cuda")
    for s in range(2):
        a, b = q_starts[s], q_starts[s + 1]
        if not 0 <= a <= b <= T:
            continue
        covered[a:b] = True
        o, le, to, tl = ref.attend(q[a:b], k[s], v[s], D ** -0.5)
        ref.check(out[a:b], o, to, f"out {s}")
        ref.check(lse[a:b], le, tl, f"lse {s}")
    assert bool((out[~covered] == 7.0).all()) and bool((lse[~covered] == 7.0).all())
    assert call([0, 20, T])[2] == 0
