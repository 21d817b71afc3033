"""GPU tests of rows whose logits outgrow the scale that their first logits set:
the new scale, the rescaled sum and output, in either half of a block, seen
whole or masked, in whole rows, parts and shared prefixes, for both types and
head sizes, against the definition in 64 bits."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_reference as ref  # noqa: E402
from test_gpu_attention import BF, HF, gen_of, ints, starts  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


# log2 of the weights of the keys, 64 at a time (the first 16 keys: 0).  A new
# scale is due where 64 weights sum up to more than 2^15 of the scale in use,
# that is from about 9 above it on: in the halves 3, 6, 8 and 9; the halves
# between stay below that with sums that still count beside the next.
STAIRS = [8.0, 8.0, 8.6, 9.8, 17.5, 18.2, 19.6, 28.0, 29.4, 38.8, 38.8, 46.0, 46.0, 46.4]
PERIOD = 64 * len(STAIRS)
# ends right after, before and amid each of them
ENDS = [17, 64, 100, 192, 230, 256, 257, 320, 448, 500, 576, 577, 640, 700, 896, 1100]


def level(n):
    at = torch.arange(n, device="cuda") % PERIOD
    return torch.where(at < 16, 0.0, torch.tensor(STAIRS, device="cuda")[at // 64])


def stair_keys(gen, Hkv, n, D, dtype, sign):
    """Keys whose products with queries of about ones have these levels, scale 1 / sqrt(D)."""
    k = (level(n) * 0.6931 / D ** 0.5)[None, :, None] + 0.2 * torch.randn(Hkv, n, D, generator=gen, device="cuda")
    return (sign * k).to(dtype)


def stair_queries(gen, T, Hq, D, dtype):
    return (1 + 0.02 * torch.randn(T, Hq, D, generator=gen, device="cuda")).to(dtype)


def values(gen, Hkv, n, D, dtype):
    return torch.randn(Hkv, n, D, generator=gen, device="cuda").to(dtype)


def paged(gen, k, v, page):
    """A cache of these lists of [Hkv, n, D], its unused rows NaN, and the page table."""
    Hkv, _, D = k[0].shape
    need = [(x.shape[1] + page - 1) // page for x in k]
    order = torch.randperm(sum(need), generator=gen, device="cuda").tolist()
    kc = torch.full((sum(need), Hkv, page, D), float("nan"), dtype=k[0].dtype, device="cuda")
    vc = kc.clone()
    table = torch.full((len(k), max(need)), -1, dtype=torch.int32)
    at = 0
    for s in range(len(k)):
        for j in range(need[s]):
            rows = slice(j * page, min((j + 1) * page, k[s].shape[1]))
            p = order[at]
            at += 1
            table[s, j] = p
            kc[p, :, :rows.stop - rows.start], vc[p, :, :rows.stop - rows.start] = k[s][:, rows], v[s][:, rows]
    return kc, vc, table.cuda()


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_prefill(dtype, D, page, causal, sign):
    Hq, Hkv, rows = 8, 4, 40
    g = gen_of(11)
    q = stair_queries(g, rows * len(ENDS), Hq, D, dtype)
    k = [stair_keys(g, Hkv, n, D, dtype, sign) for n in ENDS]
    v = [values(g, Hkv, n, D, dtype) for n in ENDS]
    qs = starts([rows] * len(ENDS))
    lse = torch.full((q.shape[0], Hq), 7.0, device="cuda")
    scale = sign * D ** -0.5
    ws = moe.alloc_attn_workspace(q.shape[0], len(ENDS), Hq, Hkv, D)
    if page:
        kc, vc, table = paged(g, k, v, page)
        out = moe.attn_prefill_paged(q, kc, vc, table, qs, ints(ENDS), causal=causal, scale=scale, lse=lse, workspace=ws)
    else:
        kk, vv = (torch.cat(x, 1).transpose(0, 1).contiguous() for x in (k, v))
        out = moe.attn_prefill(q, kk, vv, qs, starts(ENDS), causal=causal, scale=scale, lse=lse, workspace=ws)
    assert moe.read_status(ws) == 0
    for s, n in enumerate(ENDS):
        at = slice(s * rows, (s + 1) * rows)
        seen = ref.causal(rows, n, "cuda") if causal else None
        o, le, to, tl = ref.attend(q[at], k[s], v[s], scale, seen)
        ref.check(out[at], o, to, f"out, {n} keys")
        ref.check(lse[at], le, tl, f"lse, {n} keys")


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,n", [(9, 5000), (70, 2900), (1, 1100)])
def test_prefill_split(dtype, D, rows, n):
    # keys split over blocks: every part climbs stairs of its own
    Hq, Hkv = 8, 1
    g = gen_of(12)
    q = stair_queries(g, rows, Hq, D, dtype)
    k, v = stair_keys(g, Hkv, n, D, dtype, 1), values(g, Hkv, n, D, dtype)
    lse = torch.empty(rows, Hq, device="cuda")
    out = moe.attn_prefill(q, k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous(), starts([rows]), starts([n]),
                           lse=lse)
    o, le, to, tl = ref.attend(q, k, v, D ** -0.5, ref.causal(rows, n, "cuda"))
    ref.check(out, o, to, "out")
    ref.check(lse, le, tl, "lse")


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [0, 700, 5000])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (24, 1)])
def test_decode(dtype, D, prefix, Hq, Hkv):
    page = 16
    g = gen_of(13)
    lens = [17, 256, 0, 577, 3000]
    q = stair_queries(g, len(lens), Hq, D, dtype)
    k = [stair_keys(g, Hkv, n, D, dtype, 1) for n in lens + [prefix]]
    v = [values(g, Hkv, n, D, dtype) for n in lens + [prefix]]
    kc, vc, table = paged(g, k, v, page)
    lse = torch.empty(len(lens), Hq, device="cuda")
    out = moe.attn_decode(q, kc, vc, table[:-1].contiguous(), ints(lens), table[-1] if prefix else None, prefix, lse=lse)
    for b, n in enumerate(lens):
        kk, vv = torch.cat([k[-1], k[b]], 1), torch.cat([v[-1], v[b]], 1)
        o, le, to, tl = ref.attend(q[b:b + 1], kk, vv, D ** -0.5)
        ref.check(out[b:b + 1], o, to, f"out, {n} own keys")
        ref.check(lse[b:b + 1], le, tl, f"lse, {n} own keys")
