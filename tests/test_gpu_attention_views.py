"""GPU tests of attention on other layouts than the usual: page tables much
wider than any sequence needs, head-major views, sequences by themselves, and
the status of calls with bad lengths and pages."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_reference as ref  # noqa: E402
import test_gpu_attention as base  # noqa: E402
from test_gpu_attention import BF, HF, MOE_ERR_DEVICE, gen_of, ints, rand, starts  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


def widened(table, pages):
    """The table with room for this many pages a sequence; the entries past the sequences' own name no page."""
    wide = torch.full((table.shape[0], pages), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = torch.where((table >= 0) & (table < (1 << 29)), table, -1)
    return wide


@pytest.mark.parametrize("q_lens,kv_lens", [([64], [200]), ([1], [1]), ([30, 1, 0, 90], [700, 0, 12, 2000])],
                         ids=lambda v: "-".join(map(str, v)))
@pytest.mark.parametrize("page", [16, 128])
def test_wide_tables(q_lens, kv_lens, page):
    # room for 131,072 keys a sequence
    Hq, Hkv, D = 32, 4, 128
    kc, vc, table, _ = base.page_pool(kv_lens, page, Hkv, D, BF, 21)
    wide = widened(table, 131072 // page)
    q = rand(gen_of(22), sum(q_lens), Hq, D, mul=2.5)
    keys = [[ref.paged(c, table[s, :(n + page - 1) // page], n) for c in (kc, vc)] for s, n in enumerate(kv_lens)]
    lse = torch.full((q.shape[0], Hq), 7.0, device="cuda")
    ws = moe.alloc_attn_workspace(q.shape[0], len(q_lens), Hq, Hkv, D)
    out = moe.attn_prefill_paged(q, kc, vc, wide, starts(q_lens), ints(kv_lens), lse=lse, workspace=ws)
    assert moe.read_status(ws) == 0
    o, le, to, tl = base.prefill_reference(q, q_lens, lambda s: keys[s], True, D ** -0.5)
    ref.check(out, o, to, "out")
    ref.check(lse, le, tl, "lse")
    rows = rand(gen_of(23), len(kv_lens), Hq, D, mul=2.5)
    ws = moe.alloc_attn_workspace(len(kv_lens), len(kv_lens), Hq, Hkv, D)
    out = moe.attn_decode(rows, kc, vc, wide, ints(kv_lens), workspace=ws)
    assert moe.read_status(ws) == 0
    for b, (k, v) in enumerate(keys):
        o, _, to, _ = ref.attend(rows[b:b + 1], k, v, D ** -0.5)
        ref.check(out[b:b + 1], o, to, f"decode {b}")


def head_major(gen, T, heads, D, dtype, mul=1.0):
    """[T, heads, D] whose heads lie one after the other."""
    return rand(gen, heads, T + 3, D, dtype=dtype, mul=mul)[:, :T].transpose(0, 1)


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, BF), (6, 6, 64, HF), (14, 2, 64, BF)])
def test_head_major_views(Hq, Hkv, D, dtype):
    q_lens, kv_lens, g = [130, 1, 70], [130, 600, 300], gen_of(31)
    q = head_major(g, sum(q_lens), Hq, D, dtype, 2.5)
    k, v = head_major(g, sum(kv_lens), Hkv, D, dtype), head_major(g, sum(kv_lens), Hkv, D, dtype)
    at = [int(x) for x in starts(kv_lens)]
    out = moe.attn_prefill(q, k, v, starts(q_lens), starts(kv_lens))
    o, _, to, _ = base.prefill_reference(q, q_lens, lambda s: (k[at[s]:at[s + 1]].transpose(0, 1),
                                                              v[at[s]:at[s + 1]].transpose(0, 1)), True, D ** -0.5)
    ref.check(out, o, to, "prefill")
    kc, vc, table, _ = base.page_pool([40, 90], 16, Hkv, D, dtype, 32)
    rows = head_major(g, 2, Hq, D, dtype, 2.5)
    out = moe.attn_decode(rows, kc, vc, table, ints([40, 90]))
    o, _, to, _ = base.decode_reference(rows, kc, vc, table, None, [40, 90], 0, 16, D ** -0.5)
    ref.check(out, o, to, "decode")
    T = 50
    q, k, v = (head_major(g, T, h, D, dtype) for h in (Hq, Hkv, Hkv))
    table = moe.rope_table(100, D)
    slots = torch.randperm(64, generator=g, device="cuda")[:T].to(torch.int32)
    kc, vc = rand(g, 4, Hkv, 16, D, dtype=dtype), rand(g, 4, Hkv, 16, D, dtype=dtype)
    kc0, vc0 = kc.clone(), vc.clone()
    pos = ints(list(range(T)))
    out = moe.rope_append(q, k, v, table, pos, slots, kc, vc)
    base.rope_check(q, k, v, table, pos, slots, kc0, vc0, kc, vc, None, None, D, False, out)


def test_a_sequence_alone_and_among_others():
    # enough heads that no call splits its keys: the same blocks in the same order, the same bits
    lens, H, D = [300, 900, 17, 260], 80, 64
    q, k, v = base.packed_case(lens, lens, H, H, D, BF, 34)
    at = [int(x) for x in starts(lens)]
    together = moe.attn_prefill(q, k, v, starts(lens), starts(lens))
    for s in (0, 1, 3):
        rows = slice(at[s], at[s + 1])
        alone = moe.attn_prefill(q[rows], k[rows], v[rows], starts([lens[s]]), starts([lens[s]]))
        assert torch.equal(alone, together[rows])


def test_status_of_bad_lengths_and_pages_of_long_sequences():
    q_lens, kv_lens, Hq, Hkv, D, page = [300, 17, 1, 512], [4100, 3500, 4000, 512], 32, 4, 128, 16
    kc, vc, table, _ = base.page_pool(kv_lens, page, Hkv, D, BF, 21)
    q = rand(gen_of(22), sum(q_lens), Hq, D, mul=2.5)
    ws = moe.alloc_attn_workspace(q.shape[0], 4, Hq, Hkv, D)
    bad = table.clone()
    bad[2, 7] = 1 << 29
    for t, lens, status in ((table, kv_lens, 0), (table, [4100, 1 << 30, 4000, 512], MOE_ERR_DEVICE),
                            (table, [4100, 3500, -1, 512], MOE_ERR_DEVICE), (bad, kv_lens, MOE_ERR_DEVICE),
                            (table, kv_lens, 0)):
        moe.attn_prefill_paged(q, kc, vc, t, starts(q_lens), ints(lens), workspace=ws)
        assert moe.read_status(ws) == status
