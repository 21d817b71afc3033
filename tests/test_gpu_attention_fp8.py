"""GPU tests of attention over a paged cache in 8 bits against the definition
in 64 bits: prompts, single tokens, shared prefixes."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_reference as ref  # noqa: E402
import cache8_reference as c8  # noqa: E402
import test_gpu_attention_waits as waits  # noqa: E402
from test_gpu_attention import BF, HF, gen_of, ints, rand, starts  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu

MOE_ERR_DEVICE = -5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


def pool(lens, page, Hkv, D, seed, prefix=0, spread=4):
    """A cache whose unused rows and pages hold NaN codes and whose scales of unused blocks are anything, page lists
    with their unused entries out of range, and the prefix's pages.  Scales of blocks differ by up to 2^(2 spread)."""
    g = gen_of(seed)
    need = [(n + page - 1) // page for n in lens]
    extra = (prefix + page - 1) // page
    total = sum(need) + extra + 3
    kc, vc, sc = moe.alloc_fp8_cache(total, Hkv, page, D)
    for c in (kc, vc):
        x = torch.randn(c.shape, generator=g, device="cuda") * 100
        c.copy_(x.clamp(-448, 448).to(c8.F8))
    # keys as a norm leaves them, about 1 in size; values of any
    sc[..., 0] = 2.0 ** -7 * torch.exp2(torch.randint(-1, 2, sc.shape[:3], generator=g, device="cuda").float())
    sc[..., 1] = 2.0 ** -7 * torch.exp2(torch.randint(-spread, spread + 1, sc.shape[:3], generator=g, device="cuda").float())
    order = torch.randperm(total, generator=g, device="cuda").tolist()
    table = torch.full((len(lens), max(max(need, default=0), 1) + 1), 1 << 30, dtype=torch.int32)
    used = torch.zeros(total, page, dtype=torch.bool)
    at = 0
    for s, n in enumerate(lens):
        for j in range(need[s]):
            table[s, j] = order[at]
            used[order[at], :min(page, n - j * page)] = True
            at += 1
    pre = order[at:at + extra]
    for j, p in enumerate(pre):
        used[p, :min(page, prefix - j * page)] = True
    junk = ~used.cuda()
    for c in (kc, vc):
        c.view(torch.uint8).masked_fill_(junk[:, None, :, None], 0x7f)               # NaN
    blocks = used.view(total, page // 16, 16).any(-1).cuda()
    sc.copy_(torch.where(blocks[:, None, :, None], sc, torch.full_like(sc, float("nan"))))
    return kc, vc, sc, table.cuda(), ints(pre) if prefix else None


def rows(kc, vc, sc, pages, n):
    page = kc.shape[2]
    ids = pages[:(n + page - 1) // page]
    return c8.rows(kc, sc, 0, ids, n), c8.rows(vc, sc, 1, ids, n)


def prefill_check(q, q_lens, kv_lens, kc, vc, sc, table, causal, scale, out, lse):
    at = 0
    for s, n in enumerate(q_lens):
        k, v = rows(kc, vc, sc, table[s], kv_lens[s])
        seen = ref.causal(n, kv_lens[s], q.device) if causal else None
        o, le, to, tl = c8.attend(q[at:at + n], k, v, scale, seen, parts=True)
        ref.check(out[at:at + n], o, to, f"out of sequence {s}")
        ref.check(lse[at:at + n], le, tl, f"lse of sequence {s}")
        at += n


PREFILL = [
    # q_lens, kv_lens, Hq, Hkv, D, causal, page, dtype
    ([1], [1], 8, 2, 128, True, 16, BF),
    ([1, 40, 130], [1, 200, 130], 8, 2, 128, True, 16, BF),
    ([1, 40, 130], [1, 200, 130], 8, 2, 128, True, 16, HF),
    ([64, 3], [1000, 515], 8, 1, 128, True, 32, BF),
    ([100], [777], 4, 4, 64, False, 64, HF),
    ([129, 0, 31], [129, 50, 1031], 7, 1, 64, True, 128, BF),
    ([50, 60], [300, 20], 6, 3, 128, True, 256, HF),                 # more rows than keys: rows that see none
    ([1, 2, 3, 4], [3000, 0, 5, 4], 32, 4, 128, True, 16, BF),
    ([8], [9000], 8, 1, 128, True, 64, BF),
    ([300, 17, 1, 512], [4100, 3500, 4000, 512], 32, 4, 128, True, 16, BF),
    ([1400], [5001], 16, 8, 64, True, 64, HF),
    ([150, 400], [60, 3500], 48, 4, 128, True, 128, BF),
    ([5, 3], [300, 129], 128, 1, 64, True, 16, BF),                  # every head on one key-value head
    ([20] * 70, [20] * 70, 4, 2, 64, True, 16, BF),
    ([200, 90], [4000, 0], 16, 16, 64, False, 32, HF),
]


@pytest.mark.parametrize("case", PREFILL, ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}-p{c[6]}-{sum(c[0])}-{sum(c[1])}-{str(c[7])[6:]}")
def test_prefill(case):
    q_lens, kv_lens, Hq, Hkv, D, causal, page, dtype = case
    kc, vc, sc, table, _ = pool(kv_lens, page, Hkv, D, 31)
    q = rand(gen_of(32), sum(q_lens), Hq, D + 8, dtype=dtype, mul=2.5)[..., :D]
    lse = torch.full((q.shape[0], Hq), 7.0, device="cuda")
    ws = moe.alloc_attn_workspace(q.shape[0], len(q_lens), Hq, Hkv, D)

    def call():
        return moe.attn_prefill_paged_fp8(q, kc, vc, sc, table, starts(q_lens), ints(kv_lens), causal=causal, lse=lse,
                                          workspace=ws)
    out = call()
    assert moe.read_status(ws) == 0
    prefill_check(q, q_lens, kv_lens, kc, vc, sc, table, causal, D ** -0.5, out, lse)
    assert torch.equal(out, call())


DECODE = [
    # kv_lens, prefix, Hq, Hkv, D, page, dtype
    ([1], 0, 8, 1, 128, 16, BF),
    ([0, 1, 15, 16, 17, 129], 0, 8, 2, 128, 16, BF),
    ([0, 1, 15, 16, 17, 129], 0, 16, 2, 64, 32, HF),
    ([300, 7, 4000], 0, 32, 4, 128, 16, BF),
    ([300, 7, 4000], 0, 48, 2, 128, 64, HF),                         # 24 heads on one: two units
    ([300, 7, 4000], 0, 14, 1, 64, 128, BF),
    ([30000], 0, 8, 2, 64, 64, BF),
    ([30000], 0, 4, 4, 128, 256, HF),
    ([50] * 300, 0, 8, 2, 128, 16, BF),
    ([0, 40, 700], 1000, 8, 2, 128, 16, BF),
    ([0, 40, 700], 1000, 8, 2, 128, 16, HF),
    ([0, 0], 129, 6, 3, 64, 32, BF),
    ([5, 3000] * 20, 2000, 32, 4, 128, 16, BF),
    ([50000, 40000], 100, 16, 2, 64, 64, BF),                        # short prefix, long own keys
]


def decode_check(q, kv_lens, prefix, kc, vc, sc, table, pre, scale, out, lse, rows_of=None):
    for b, n in enumerate(kv_lens):
        k, v = rows(kc, vc, sc, table[b], n)
        if prefix:
            pk, pv = rows(kc, vc, sc, pre, prefix)
            k, v = torch.cat([pk, k], 1), torch.cat([pv, v], 1)
        o, le, to, tl = c8.attend(q[b:b + 1], k, v, scale)
        ref.check(out[b:b + 1], o, to, f"out of row {b}")
        ref.check(lse[b:b + 1], le, tl, f"lse of row {b}")


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}-p{c[5]}-{len(c[0])}x{max(c[0])}-pre{c[1]}-{str(c[6])[6:]}")
def test_decode(case):
    kv_lens, prefix, Hq, Hkv, D, page, dtype = case
    kc, vc, sc, table, pre = pool(kv_lens, page, Hkv, D, 41, prefix)
    B = len(kv_lens)
    q = rand(gen_of(42), B, Hq, D, dtype=dtype, mul=2.5)
    lse = torch.full((B, Hq), 7.0, device="cuda")
    ws = moe.alloc_attn_workspace(B, B, Hq, Hkv, D)

    def call():
        return moe.attn_decode_fp8(q, kc, vc, sc, table, ints(kv_lens), pre, prefix, lse=lse, workspace=ws)
    out = call()
    assert moe.read_status(ws) == 0
    decode_check(q, kv_lens, prefix, kc, vc, sc, table, pre, D ** -0.5, out, lse)
    assert torch.equal(out, call())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-33, 2.0])
def test_scales_of_logits(scale, dtype):
    kv_lens, q_lens, Hq, Hkv, D, page = [70, 300], [5, 40], 8, 2, 128, 16
    kc, vc, sc, table, _ = pool(kv_lens, page, Hkv, D, 51)
    q = rand(gen_of(52), 45, Hq, D, dtype=dtype)
    lse = torch.empty(45, Hq, device="cuda")
    out = moe.attn_prefill_paged_fp8(q, kc, vc, sc, table, starts(q_lens), ints(kv_lens), scale=scale, lse=lse)
    prefill_check(q, q_lens, kv_lens, kc, vc, sc, table, True, scale, out, lse)
    out = moe.attn_decode_fp8(q[:2], kc, vc, sc, table, ints(kv_lens), scale=scale, lse=lse[:2])
    decode_check(q[:2], kv_lens, 0, kc, vc, sc, table, None, scale, out, lse[:2])


@pytest.mark.parametrize("dtype", [BF, HF])
def test_scales_far_apart(dtype):
    """Values of 2^-24 beside values of 2^7 scales, a sink of small values with most of the weight, blocks of zeros,
    and keys whose scales make a row outgrow its first scale."""
    kv_lens, Hq, Hkv, D, page = [400, 65], 4, 1, 128, 16
    kc, vc, sc, table, _ = pool(kv_lens, page, Hkv, D, 61)
    q = rand(gen_of(62), 2, Hq, D, dtype=dtype)
    sc[..., 1] = 2.0 ** -7
    first = [int(x) for x in table[0, :25]]
    sc[first[3], 0, 0, 1] = 2.0 ** -24
    sc[first[9], 0, 0, 1] = 2.0 ** 7
    sc[first[12], 0, 0, 0] = 2.0 ** -4                    # large logits later on
    sc[first[20], 0, 0, 0] = 2.0 ** -3
    vc.view(torch.uint8)[first[5]] = 0
    sink = int(table[1, 0])
    sc[sink, 0, 0, 1] = 2.0 ** -24
    kc.view(torch.uint8)[sink, 0, 0] = (q[1, 0].float() * 40).clamp(-448, 448).to(c8.F8).view(torch.uint8)
    lse = torch.empty(2, Hq, device="cuda")
    out = moe.attn_decode_fp8(q, kc, vc, sc, table, ints(kv_lens), lse=lse)
    decode_check(q, kv_lens, 0, kc, vc, sc, table, None, D ** -0.5, out, lse)
    out = moe.attn_prefill_paged_fp8(q, kc, vc, sc, table, ints([0, 1, 2]), ints(kv_lens), lse=lse)
    prefill_check(q, [1, 1], kv_lens, kc, vc, sc, table, True, D ** -0.5, out, lse)


@pytest.mark.parametrize("D,dtype", [(64, BF), (64, HF), (128, BF), (128, HF)])
def test_scales_and_queries_far_apart(D, dtype):
    """Scales of values from one end of their range to the other within a tile, and rows of queries with one element
    that is 2^6 to 2^12 times the others."""
    kv_lens, q_lens, Hq, Hkv, page = [400, 1000], [90, 1], 8, 2, 32
    kc, vc, sc, table, _ = pool(kv_lens, page, Hkv, D, 61, spread=14)
    q = rand(gen_of(62), sum(q_lens), Hq, D, dtype=dtype)
    high = torch.arange(Hq, device="cuda")
    q[:, high, high * 5] = 2.0 ** (6 + high % 7).to(dtype)
    scale = 0.25 * D ** -0.5
    lse = torch.empty(q.shape[0], Hq, device="cuda")
    out = moe.attn_prefill_paged_fp8(q, kc, vc, sc, table, starts(q_lens), ints(kv_lens), scale=scale, lse=lse)
    prefill_check(q, q_lens, kv_lens, kc, vc, sc, table, True, scale, out, lse)
    out = moe.attn_decode_fp8(q[-2:], kc, vc, sc, table, ints(kv_lens), scale=scale, lse=lse[-2:])
    decode_check(q[-2:], kv_lens, 0, kc, vc, sc, table, None, scale, out, lse[-2:])


@pytest.mark.parametrize("mul", [1e-30, 1e-6, 1e6, 1e30])
def test_bf16_queries_of_any_size(mul):
    """Beyond f16's range on either side; the logits brought back by the scale."""
    kv_lens, Hq, Hkv, D, page = [300, 20], 8, 2, 64, 16
    kc, vc, sc, table, _ = pool(kv_lens, page, Hkv, D, 71)
    q = (torch.randn(2, Hq, D, generator=gen_of(72), device="cuda") * mul).to(BF)
    q[0, 3, 5:] = 0
    lse = torch.empty(2, Hq, device="cuda")
    scale = 0.3 / mul if mul != 1e-30 else 1e29
    out = moe.attn_decode_fp8(q, kc, vc, sc, table, ints(kv_lens), scale=scale, lse=lse)
    decode_check(q, kv_lens, 0, kc, vc, sc, table, None, scale, out, lse)
    out = moe.attn_prefill_paged_fp8(q, kc, vc, sc, table, ints([0, 1, 2]), ints(kv_lens), scale=scale, lse=lse)
    prefill_check(q, [1, 1], kv_lens, kc, vc, sc, table, True, scale, out, lse)


def test_nan_stays_with_its_rows():
    kv_lens, q_lens, Hq, Hkv, D, page = [100, 100, 100], [3, 3, 3], 4, 2, 64, 16
    kc, vc, sc, table, _ = pool(kv_lens, page, Hkv, D, 81)
    kc.view(torch.uint8)[int(table[1, 2]), 0, 5, 7] = 0x7f            # a key of head 0 of sequence 1
    vc.view(torch.uint8)[int(table[2, 1]), 1, 4, 9] = 0xff            # a value of head 1 of sequence 2
    q = rand(gen_of(82), 9, Hq, D)

    def check(o):
        o = o.isnan().view(3, -1, 2, 2, D)                            # sequence, row, key-value head, head of it
        assert not o[0].any() and o[1, :, 0].all() and not o[1, :, 1].any()
        assert o[2, :, 1, :, 9].all() and not o[2, :, 0].any() and int(o[2].sum()) == o.shape[1] * 2
    check(moe.attn_prefill_paged_fp8(q, kc, vc, sc, table, starts(q_lens), ints(kv_lens), causal=False))
    check(moe.attn_decode_fp8(q[::3].contiguous(), kc, vc, sc, table, ints(kv_lens)))


@pytest.mark.parametrize("D,dtype", [(64, BF), (64, HF), (128, BF), (128, HF)])
def test_an_infinite_query_stays_with_its_head(D, dtype):
    kv_lens, q_lens, Hq, Hkv, page = [300, 40], [70, 40], 8, 2, 16
    kc, vc, sc, table, _ = pool(kv_lens, page, Hkv, D, 83)
    q = rand(gen_of(84), sum(q_lens), Hq, D, dtype=dtype)
    q[3] = 0                                                      # rows of zeros are rows like others

    def call():
        return moe.attn_prefill_paged_fp8(q, kc, vc, sc, table, starts(q_lens), ints(kv_lens))
    want = call()
    assert not want.isnan().any()
    for at, x in ((5, float("inf")), (33, -float("inf")), (80, float("nan"))):
        q[at, 2, at % D] = x
    got = call()
    for at in (5, 33, 80):
        assert got[at, 2].isnan().all()
        got[at, 2] = want[at, 2]
    assert torch.equal(got, want)


def test_what_is_out_of_range_is_reported():
    kv_lens, q_lens, Hq, Hkv, D, page = [100, 50, 70], [3, 5, 2], 4, 2, 64, 16
    kc, vc, sc, table, pre = pool(kv_lens, page, Hkv, D, 91, prefix=40)
    q = rand(gen_of(92), 10, Hq, D)
    ws = moe.alloc_attn_workspace(10, 3, Hq, Hkv, D)

    def prefill(table, lens):
        out = moe.attn_prefill_paged_fp8(q, kc, vc, sc, table, starts(q_lens), ints(lens), workspace=ws)
        return out, moe.read_status(ws)

    def decode(table, lens, pre):
        out = moe.attn_decode_fp8(q[:3], kc, vc, sc, table, ints(lens), pre, 40, workspace=ws)
        return out, moe.read_status(ws)
    clean, status = prefill(table, kv_lens)
    dclean, dstatus = decode(table, kv_lens, pre)
    assert status == 0 and dstatus == 0
    for bad in (-1, kc.shape[0]):
        t = table.clone()
        t[1, 2] = bad
        out, status = prefill(t, kv_lens)
        assert status == MOE_ERR_DEVICE and torch.equal(out[:3], clean[:3]) and torch.equal(out[8:], clean[8:])
        out, status = decode(t, kv_lens, pre)
        assert status == MOE_ERR_DEVICE and torch.equal(out[::2], dclean[::2])
        p = pre.clone()
        p[1] = bad
        assert decode(table, kv_lens, p)[1] == MOE_ERR_DEVICE
    for bad in (-1, 1 << 20):
        lens = [100, bad, 70]
        assert prefill(table, lens)[1] == MOE_ERR_DEVICE and decode(table, lens, pre)[1] == MOE_ERR_DEVICE
    assert prefill(table, kv_lens)[1] == 0 and decode(table, kv_lens, pre)[1] == 0


def test_captured_twice_with_a_workspace_each():
    kv_lens, Hq, Hkv, D, page = [700, 3000, 20], 8, 2, 128, 16
    kc, vc, sc, table, pre = pool(kv_lens, page, Hkv, D, 95, prefix=300)
    q = rand(gen_of(96), 3, Hq, D)
    outs = [torch.empty_like(q) for _ in range(2)]
    spaces = [moe.alloc_attn_workspace(3, 3, Hq, Hkv, D) for _ in range(2)]
    n = ints(kv_lens)
    want = moe.attn_decode_fp8(q, kc, vc, sc, table, n, pre, 300)
    graphs = []
    for o, w in zip(outs, spaces):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            moe.attn_decode_fp8(q, kc, vc, sc, table, n, pre, 300, out=o, workspace=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


# (heads of 64 have eight stages: the few blocks of an item here wait for none to be given back; decode over codes waits
# for copies alone, which always end)
@pytest.mark.parametrize("wait,D,dtype", [(w, 128, BF) for w in range(2, 12)] +
                         [(w, 64, HF) for w in range(2, 12) if w != 3])
def test_waits_that_give_up(wait, D, dtype):
    """As in the tests of the other waits: a barrier that never completes ends the call with a report, and the next
    call on the workspace is right."""
    page, Hq, Hkv = 16, 8, 2
    # more items than SMs where the wait is for the next one, and rows that outgrow their scale for the half block's
    n, n_q, keys = (160, 50, 300) if wait == 11 else (2, 60, 900)
    Hq, Hkv = (4, 1) if wait == 11 else (Hq, Hkv)
    kc, vc, sc, table, _ = pool([keys] * n, page, Hkv, D, 99)
    q = rand(gen_of(98), n * n_q, Hq, D, dtype=dtype)
    q[..., 0] = 4
    for s in range(n):
        kc.view(torch.uint8)[int(table[s, 6]), :, 4, 0] = 0x7e        # key 100 of the first block: 448
        sc[int(table[s, 6]), :, 0, 0] = 2.0 ** -2
    ws = moe.alloc_attn_workspace(n * n_q, n, Hq, Hkv, D)
    waits.times_out(lambda: moe.attn_prefill_paged_fp8(q, kc, vc, sc, table, starts([n_q] * n), ints([keys] * n),
                                                       causal=False, workspace=ws), ws, wait, junk=wait != 11)
