"""GPU tests of attention over keys whose logits are -inf (an infinity in a key,
or a product past fp32): such a key weighs nothing, as if it were not there, and
a row whose keys are all of this kind has out = 0 and lse = -inf."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_reference as ref  # noqa: E402
import test_gpu_attention as base  # noqa: E402
from test_gpu_attention import BF, HF, gen_of, ints, rand, starts  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


# keys whose logits are -inf, of n
GONE = {
    "first16": lambda n: range(min(16, n)),
    "first100": lambda n: range(min(100, n)),
    "first block": lambda n: range(min(128, n)),
    "first block and 16": lambda n: range(min(144, n)),
    "all but the last": lambda n: range(n - 1),
    "second block": lambda n: range(128, min(256, n)),
    "every third": lambda n: range(0, n, 3),
    "all": lambda n: range(n),
}


def spoil(keys, at, scale, overflow):
    """Element 0 of keys [Hkv, n, D] at these places, on the even heads: times q's
    element 0 (at least 1) and the scale a logit of -inf."""
    value = (-3e38 if overflow else -math.inf) * (1 if scale > 0 else -1)
    keys[::2, list(at), 0] = value


def queries(gen, T, Hq, D, dtype):
    q = rand(gen, T, Hq, D, dtype=dtype, mul=2.5)
    q[..., 0] = q[..., 0].abs() + (16 if dtype == BF else 1)
    return q


def want(q, k, v, gone, scale, causal):
    """k before it was spoilt; keys that weigh nothing count as not seen."""
    n, m = q.shape[0], k.shape[1]
    group = q.shape[1] // k.shape[0]
    seen = ref.causal(n, m, q.device) if causal else torch.ones(n, m, dtype=torch.bool, device=q.device)
    fewer = seen.clone()
    fewer[:, list(gone)] = False
    res = [ref.attend(q, k, v, scale, s) for s in (fewer, seen)]
    spoilt = torch.arange(q.shape[1], device=q.device) // group % 2 == 0
    return [torch.where(spoilt[None, :, None] if x.dim() == 3 else spoilt[None, :], x, y) for x, y in zip(*res)]


PREFILL = [
    # rows, keys, Hq, Hkv, D, causal, page (0: packed), dtype, scale
    (200, 128, 4, 2, 64, False, 0, HF, 0.125),
    (200, 256, 4, 2, 128, False, 0, BF, 0.09),
    (70, 700, 12, 12, 64, False, 0, HF, 0.125),
    (300, 300, 8, 2, 128, True, 0, BF, 0.09),
    (64, 700, 14, 2, 128, True, 16, BF, 0.09),
    (130, 400, 4, 2, 64, True, 128, HF, -0.125),
    (9, 4000, 4, 2, 128, False, 0, BF, -0.09),          # keys split over blocks
    (20, 5000, 8, 2, 64, True, 32, BF, 0.125),
]


@pytest.mark.parametrize("gone", GONE)
@pytest.mark.parametrize("case", PREFILL, ids=lambda c: "-".join(map(str, c)))
def test_prefill(case, gone):
    n, m, Hq, Hkv, D, causal, page, dtype, scale = case
    at = GONE[gone](m)
    q = queries(gen_of(3), n, Hq, D, dtype)
    lse = torch.full((n, Hq), 7.0, device="cuda")
    if page:
        kc, vc, table, _ = base.page_pool([m], page, Hkv, D, dtype, 5)
        pages = table[0, :(m + page - 1) // page]
        k, v = ref.paged(kc, pages, m).clone(), ref.paged(vc, pages, m)
        bad = k.clone()
        spoil(bad, at, scale, overflow=dtype == BF)
        for j, p in enumerate(pages.tolist()):
            rows = bad[:, j * page:(j + 1) * page]
            kc[p, :, :rows.shape[1]] = rows
        out = moe.attn_prefill_paged(q, kc, vc, table, starts([n]), ints([m]), causal=causal, scale=scale, lse=lse)
    else:
        g = gen_of(4)
        k, v = rand(g, Hkv, m, D, dtype=dtype), rand(g, Hkv, m, D, dtype=dtype)
        bad = k.clone()
        spoil(bad, at, scale, overflow=dtype == BF)
        out = moe.attn_prefill(q, bad.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous(), starts([n]),
                               starts([m]), causal=causal, scale=scale, lse=lse)
    o, le, to, tl = want(q, k, v, at, scale, causal)
    ref.check(out, o, to, "out")
    ref.check(lse, le, tl, "lse")


DECODE = [
    # own keys, prefix, Hq, Hkv, D, page, dtype
    ([40, 0, 300], 0, 8, 2, 64, 16, HF),
    ([300, 17], 0, 48, 2, 128, 16, BF),                 # 24 heads share a key-value head
    ([9000], 0, 8, 2, 128, 64, BF),                     # joined from parts
    ([60, 0, 5000], 512, 8, 2, 128, 16, BF),
    ([0, 17], 300, 4, 2, 64, 64, HF),
]


@pytest.mark.parametrize("gone", ["first16", "first block", "every third", "all"])
@pytest.mark.parametrize("case,where", [(c, w) for c in DECODE for w in (["prefix", "own", "both"] if c[1] else ["own"])],
                         ids=lambda c: c if isinstance(c, str) else f"{c[2]}x{c[3]}x{c[4]}-B{len(c[0])}-{max(c[0])}-pre{c[1]}")
def test_decode(case, where, gone):
    kv_lens, prefix, Hq, Hkv, D, page, dtype = case
    scale = D ** -0.5
    _, kc, vc, table, pre = base.decode_case(*case)
    q = queries(gen_of(6), len(kv_lens), Hq, D, dtype)

    def break_pages(pages, n):
        k = ref.paged(kc, pages, n).clone()
        bad = k.clone()
        at = GONE[gone](n)
        spoil(bad, at, scale, overflow=dtype == BF)
        for j, p in enumerate(pages.tolist()):
            rows = bad[:, j * page:(j + 1) * page]
            kc[p, :, :rows.shape[1]] = rows
        return k, list(at)
    pk, pat = None, []
    if prefix:
        pk = ref.paged(kc, pre, prefix).clone()
        if where != "own":
            pk, pat = break_pages(pre, prefix)
    refs = [[], [], [], []]
    for b, n in enumerate(kv_lens):
        pages = table[b, :(n + page - 1) // page]
        k, at = ref.paged(kc, pages, n).clone(), []
        v = ref.paged(vc, pages, n)
        if where != "prefix":
            k, at = break_pages(pages, n)
        if prefix:
            k, v = torch.cat([pk, k], 1), torch.cat([ref.paged(vc, pre, prefix), v], 1)
            at = pat + [prefix + i for i in at]
        for r, x in zip(refs, want(q[b:b + 1], k, v, at, scale, False)):
            r.append(x)
    lse = torch.full((len(kv_lens), Hq), 7.0, device="cuda")
    ws = moe.alloc_attn_workspace(len(kv_lens), len(kv_lens), Hq, Hkv, D)
    out = moe.attn_decode(q, kc, vc, table, ints(kv_lens), pre, prefix, lse=lse, workspace=ws)
    assert moe.read_status(ws) == 0
    o, le, to, tl = (torch.cat(r) for r in refs)
    ref.check(out, o, to, "out")
    ref.check(lse, le, tl, "lse")
