"""GPU tests of the attention weight per key and of eviction by it, against
their definitions in 64 bits, and of the cache's operators used together."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_reference as ref  # noqa: E402
import cache8_reference as c8  # noqa: E402
from test_gpu_attention import BF, HF, gen_of, ints, page_pool, rand, starts  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu

MOE_ERR_DEVICE = -5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


# ------------------------------------------------------------ weight of every key
WEIGHTS = [
    # q_lens, kv_lens, Hq, Hkv, D, causal, page, dtype, entries beyond the longest
    ([1], [1], 8, 2, 128, True, 16, BF, 0),
    ([1] * 5, [0, 1, 31, 33, 700], 32, 4, 128, True, 16, BF, 3),
    ([1] * 5, [5, 64, 16, 33, 129], 7, 1, 64, True, 32, HF, 0),
    ([3, 40, 130], [3, 200, 130], 8, 2, 128, True, 16, BF, 0),
    ([100, 0, 7], [300, 50, 7], 6, 3, 64, False, 64, HF, 1),
    ([50, 60], [300, 20], 4, 4, 128, True, 256, BF, 0),              # more rows than keys
    ([64], [5000], 24, 1, 128, True, 16, BF, 8),
    ([5, 3], [300, 129], 128, 1, 64, True, 128, BF, 0),
    ([1] * 300, [40] * 300, 4, 2, 64, True, 16, BF, 0),
    ([600, 1], [600, 9000], 16, 8, 64, True, 64, BF, 5),
]


def weights_case(case, seed=3):
    q_lens, kv_lens, Hq, Hkv, D, causal, page, dtype, more = case
    kc, _, table, _ = page_pool(kv_lens, page, Hkv, D, dtype, seed)      # NaN behind the keys
    g = gen_of(seed + 1)
    q = rand(g, sum(q_lens), Hq, D + 8, dtype=dtype, mul=2.5)[..., :D]
    w = torch.rand(len(q_lens), Hkv, max(kv_lens) + more, generator=g, device="cuda")
    return q, kc, table, w


def weights_reference(q, q_lens, kv_lens, kc, table, causal, scale, lse, w):
    """The sums and the bounds on their errors (fp64).  A logit is off by D + 4 roundings of sum |q k| (attn_reference),
    its exponent by one of itself and of the log-sum and by that of 2^x, so a weight is off by that, relative; the
    sum over n rows and G heads rounds at most n G times, and once when it is added."""
    want, tol = w.double().clone(), torch.zeros_like(w, dtype=torch.float64)
    at, (Hkv, D) = 0, (kc.shape[1], kc.shape[3])
    group = q.shape[1] // Hkv
    page = kc.shape[2]
    for s, (n, m) in enumerate(zip(q_lens, kv_lens)):
        k = ref.paged(kc, table[s, :(m + page - 1) // page], m).double()
        for h in range(q.shape[1] if m else 0):
            x, kk, ll = q[at:at + n, h].double(), k[h // group], lse[at:at + n, h].double()[:, None]
            logit, mag = x @ kk.T * scale, x.abs() @ kk.abs().T * abs(scale)
            p = torch.exp(logit - ll)
            p = torch.where(ll == -math.inf, torch.zeros_like(p), p)
            if causal:
                p = torch.where(ref.causal(n, m, q.device), p, torch.zeros_like(p))
            off = (D + 4) * 2.0 ** -24 * mag + 2.0 ** -22 * (4 + mag + ll.nan_to_num(0.0, 0.0, 0.0).abs()) + n * group * 2.0 ** -24
            want[s, h // group, :m] += p.sum(0)
            tol[s, h // group, :m] += (p * off).sum(0)
        at += n
    return want, tol + 2.0 ** -23 * want.abs() + 1e-30


@pytest.mark.parametrize("case", WEIGHTS, ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}-p{c[6]}-{sum(c[0])}-{sum(c[1])}")
def test_key_weights(case):
    q_lens, kv_lens, Hq, Hkv, D, causal, page, dtype, more = case
    q, kc, table, w = weights_case(case)
    lse = torch.empty(q.shape[0], Hq, device="cuda")
    ws = moe.alloc_attn_workspace(q.shape[0], len(q_lens), Hq, Hkv, D)
    vc = torch.zeros_like(kc)
    moe.attn_prefill_paged(q, kc, vc, table, starts(q_lens), ints(kv_lens), causal=causal, lse=lse, workspace=ws)
    first = w.clone()
    got = moe.attn_key_weights(q, kc, table, starts(q_lens), ints(kv_lens), lse, w, causal=causal, workspace=ws)
    assert got is w and moe.read_status(ws) == 0
    want, tol = weights_reference(q, q_lens, kv_lens, kc, table, causal, D ** -0.5, lse, first)
    ref.check(w, want, tol, "weights")
    for s, n in enumerate(kv_lens):
        assert torch.equal(w[s, :, n:], first[s, :, n:])
    # every row that sees a key gives its heads 1 in all
    rows = [n if m else 0 for n, m in zip(q_lens, kv_lens)]
    if causal:
        rows = [min(n, m) for n, m in zip(q_lens, kv_lens)]
    given = (w - first).double().sum((1, 2))
    assert float((given - Hq * torch.tensor(rows, dtype=torch.float64, device="cuda")).abs().max()) <= 1e-3 * Hq * max(rows + [1])
    again = first.clone()
    moe.attn_key_weights(q, kc, table, starts(q_lens), ints(kv_lens), lse, again, causal=causal, workspace=ws)
    assert torch.equal(again, w)


def test_key_weights_of_rows_without_keys_and_infinite_keys():
    """A log-sum of -inf gives nothing, whatever the logits; keys that a row does not see may be anything."""
    q_lens, kv_lens, Hq, Hkv, D, page = [3, 2], [40, 20], 4, 2, 64, 16
    kc, vc, table, _ = page_pool(kv_lens, page, Hkv, D, BF, 5)
    q = rand(gen_of(6), 5, Hq, D)
    lse = torch.zeros(5, Hq, device="cuda")
    lse[1], lse[4, 2] = -math.inf, math.inf
    kc[int(table[0, 2]), :, 7] = float("nan")                # key 39: only row 2 sees it
    w = torch.zeros(2, Hkv, 40, device="cuda")
    moe.attn_key_weights(q, kc, table, starts(q_lens), ints(kv_lens), lse, w)
    assert bool(w[0, :, 39].isnan().all())
    clean = torch.where(torch.isnan(kc), torch.zeros_like(kc), kc)
    want, tol = weights_reference(q, q_lens, kv_lens, clean, table, True, D ** -0.5, lse, torch.zeros_like(w))
    ref.check(w[:, :, :39], want[:, :, :39], tol[:, :, :39], "weights")


@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_key_weights_scales(scale):
    case = WEIGHTS[3]
    q_lens, kv_lens, Hq, Hkv, D, causal, page, dtype, _ = case
    q, kc, table, w = weights_case(case)
    w.zero_()
    lse = torch.empty(q.shape[0], Hq, device="cuda")
    moe.attn_prefill_paged(q, kc, torch.zeros_like(kc), table, starts(q_lens), ints(kv_lens), scale=scale, lse=lse)
    moe.attn_key_weights(q, kc, table, starts(q_lens), ints(kv_lens), lse, w, scale=scale)
    want, tol = weights_reference(q, q_lens, kv_lens, kc, table, causal, scale, lse, torch.zeros_like(w))
    ref.check(w, want, tol, "weights")


def test_key_weights_over_shared_pages_and_capture():
    """Sequences that read the same pages have weights of their own; a captured call gives what the others do."""
    Hq, Hkv, D, page, n = 8, 2, 128, 16, 6
    kc, vc, table, _ = page_pool([200], page, Hkv, D, BF, 15)
    table = table.expand(n, -1).contiguous()
    q = rand(gen_of(16), 1, Hq, D).expand(n, -1, -1).contiguous()
    lens, lse = ints([200] * n), torch.empty(n, Hq, device="cuda")
    moe.attn_decode(q, kc, vc, table, lens, lse=lse)
    w, seq = torch.zeros(n, Hkv, 200, device="cuda"), ints(list(range(n + 1)))
    ws = moe.alloc_attn_workspace(n, n, Hq, Hkv, D)
    moe.attn_key_weights(q, kc, table, seq, lens, lse, w, workspace=ws)
    # (attn_decode splits the sequences' keys at different places: their log-sums differ in the last bits)
    want, tol = weights_reference(q, [1] * n, [200] * n, kc, table, True, D ** -0.5, lse, torch.zeros_like(w))
    ref.check(w, want, tol, "weights")
    again = torch.zeros_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.attn_key_weights(q, kc, table, seq, lens, lse, again, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, w)


def test_key_weights_report_what_is_out_of_range():
    case = ([3, 5], [100, 40], 4, 2, 64, True, 16, BF, 0)
    q, kc, table, w = weights_case(case)
    lse = torch.zeros(8, 4, device="cuda")
    ws = moe.alloc_attn_workspace(8, 2, 4, 2, 64)

    def call(table=table, qs=(0, 3, 8), lens=(100, 40), w=None):
        got = (weights_case(case)[3] if w is None else w).clone()
        moe.attn_key_weights(q, kc, table, ints(list(qs)), ints(list(lens)), lse, got, workspace=ws)
        return got, moe.read_status(ws)
    clean, status = call()
    assert status == 0
    for bad in (-1, kc.shape[0]):
        t = table.clone()
        t[1, 1] = bad
        got, status = call(t)
        assert status == MOE_ERR_DEVICE and torch.equal(got[0], clean[0])
    for lens in ((100, -1), (100, 101), (100, 1 << 20)):              # beyond the entries, beyond the table
        got, status = call(lens=lens)
        assert status == MOE_ERR_DEVICE and torch.equal(got[0], clean[0]) and torch.equal(got[1], w[1])
    assert call(qs=(0, 3, 7))[1] == MOE_ERR_DEVICE
    assert call(qs=(0, 9, 8))[1] == MOE_ERR_DEVICE
    assert call()[1] == 0


# ------------------------------------------------------------ eviction
def evict_reference(weights, n, budget, first, last):
    """Places of the keys that a head keeps."""
    if n <= budget:
        return list(range(n))
    w = [-math.inf if x != x else x for x in weights[:n]]
    nan = [x != x for x in weights[:n]]
    middle = sorted(range(first, n - last), key=lambda j: (nan[j], -w[j], j))
    return list(range(first)) + sorted(middle[:budget - first - last]) + list(range(n - last, n))


EVICT = [
    # kv_lens, budget, first, last, Hkv, D, page, dtype, kind of weights, entries beyond the longest
    ([0, 1, 7, 8, 9, 40], 8, 0, 0, 2, 64, 16, BF, "tail", 0),
    ([100, 30, 300], 40, 4, 8, 3, 128, 16, HF, "tail", 3),
    ([100, 30, 300], 40, 4, 36, 1, 64, 64, BF, "tail", 0),               # first and last alone
    ([500, 513], 128, 0, 1, 2, 128, 32, BF, "equal", 1),
    ([500, 2100], 100, 1, 0, 2, 64, 16, BF, "few", 0),                   # many of the same weight
    ([5000], 1, 0, 0, 1, 64, 128, HF, "tail", 0),
    ([5000], 4999, 2, 3, 2, 64, 256, BF, "odd", 0),                      # NaN, infinities, zeros of both signs, negative
    ([3000, 2500], 1000, 0, 5, 4, 128, 16, BF, "odd", 7),
    ([20000], 3000, 4, 64, 2, 128, 64, BF, "near", 0),                   # differ in the last bits alone
    ([60] * 1100, 20, 1, 2, 2, 64, 16, BF, "tail", 0),                   # more heads than blocks of the grid
    ([9000, 16384, 4097, 16383], 2900, 4, 64, 2, 64, 64, BF, "tail", 0),  # long, counted in registers
    ([16000, 6000, 2050], 2000, 0, 0, 1, 128, 128, HF, "odd", 9),
    ([12000, 8192], 777, 2, 1, 2, 64, 16, BF, "near", 0),
    ([16384, 3500], 1500, 1, 0, 2, 64, 256, BF, "few", 0),
    ([0, 5000, 90, 4097, 90] + [200 + 7 * i % 300 for i in range(45)], 150, 3, 9, 4, 64, 16, BF, "tail", 0),  # two to an SM
]


def evict_case(case, seed=13):
    kv_lens, budget, first, last, Hkv, D, page, dtype, kind, more = case
    out_pages = (budget + page - 1) // page
    kc, vc, table, spare = page_pool(kv_lens, page, Hkv, D, dtype, seed, extra_pages=out_pages * len(kv_lens), spare=2)
    out_table = ints(spare[:out_pages * len(kv_lens)]).view(len(kv_lens), -1)
    g = gen_of(seed + 1)
    shape = (len(kv_lens), Hkv, max(kv_lens) + more)
    w = torch.randn(shape, generator=g, device="cuda").mul(2).exp()
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "few":
        w = torch.randint(0, 3, shape, generator=g, device="cuda").float()
    elif kind == "near":
        w = (torch.randint(0, 40, shape, generator=g, device="cuda") + 0x3f800000).to(torch.int32).view(torch.float32)
    elif kind == "odd":
        w = torch.randn(shape, generator=g, device="cuda")
        pick = torch.randint(0, 8, shape, generator=g, device="cuda")
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0)):
            w[pick == i] = x
    return kc, vc, table, out_table, w


@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"{len(c[0])}x{max(c[0])}-to{c[1]}-{c[2]}-{c[3]}-{c[8]}-{c[4]}x{c[5]}-p{c[6]}")
def test_evict(case):
    kv_lens, budget, first, last, Hkv, D, page, dtype, kind, more = case
    kc, vc, table, out_table, w = evict_case(case)
    kc0, vc0, w0 = kc.clone(), vc.clone(), w.clone()
    ws = moe.alloc_attn_workspace(0, len(kv_lens), Hkv, Hkv, D)
    lens, new_w, kept = moe.kv_evict(kc, vc, table, ints(kv_lens), w, out_table, budget, keep_first=first, keep_last=last,
                                     workspace=ws)
    assert moe.read_status(ws) == 0
    assert lens.tolist() == [min(n, budget) for n in kv_lens]
    w64, bits = w0.cpu(), lambda t: t.view(torch.int16)  # noqa: E731
    kept, new_w = kept.cpu(), new_w.cpu()
    k16, v16 = kc0.clone(), vc0.clone()
    for s, n in enumerate(kv_lens):
        for h in range(Hkv):
            keep = evict_reference(w64[s, h].tolist(), n, budget, first, last)
            m = len(keep)
            assert kept[s, h].tolist() == keep + [-1] * (budget - m), (s, h)
            assert torch.equal(new_w[s, h, :m].view(torch.int32), w64[s, h, keep].view(torch.int32))
            assert bool((new_w[s, h, m:] == 0).all())
            if m:
                src, j = torch.tensor(keep, device="cuda"), torch.arange(m, device="cuda")
                at, to = table[s, src // page].long(), out_table[s, j // page].long()
                k16[to, h, j % page] = kc0[at, h, src % page]
                v16[to, h, j % page] = vc0[at, h, src % page]
    assert torch.equal(bits(kc), bits(k16)) and torch.equal(bits(vc), bits(v16))       # and nothing else changed
    assert torch.equal(w.view(torch.int32), w0.view(torch.int32))


def test_evict_reports_what_is_out_of_range():
    case = EVICT[1]
    kv_lens, budget, first, last, Hkv, D, page, dtype, kind, more = case
    kc, vc, table, out_table, w = evict_case(case)
    ws = moe.alloc_attn_workspace(0, 3, Hkv, Hkv, D)

    def call(table=table, lens=kv_lens, to=out_table):
        k, v = kc.clone(), vc.clone()
        got = moe.kv_evict(k, v, table, ints(lens), w, to, budget, keep_first=first, keep_last=last, workspace=ws)
        return got, (k, v), moe.read_status(ws)
    clean, (k0, v0), status = call()
    assert status == 0
    pages = out_table[[0, 2]].flatten().long()
    for lens in ([100, -1, 300], [100, 304, 300], [100, 1 << 20, 300]):
        got, (k, v), status = call(lens=lens)
        assert status == MOE_ERR_DEVICE and got[0].tolist() == [40, 0, 40]
        assert torch.equal(got[2][::2], clean[2][::2]) and bool((got[2][1] == -1).all())
        assert torch.equal(k[pages].view(torch.int16), k0[pages].view(torch.int16))
    for bad in (-1, kc.shape[0]):
        t, to = table.clone(), out_table.clone()
        t[1, 0] = bad
        assert call(t)[2] == MOE_ERR_DEVICE
        to[1, 0] = bad
        got, (k, v), status = call(to=to)
        assert status == MOE_ERR_DEVICE
        assert torch.equal(k[pages].view(torch.int16), k0[pages].view(torch.int16))
    assert call()[2] == 0


def test_evict_captured_and_into_given_tensors():
    case = EVICT[7]
    kv_lens, budget, first, last, Hkv, D, page, dtype, kind, more = case
    kc, vc, table, out_table, w = evict_case(case)
    n = len(kv_lens)
    out = [torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, Hkv, budget, device="cuda"),
           torch.empty(n, Hkv, budget, dtype=torch.int32, device="cuda")]
    ws, lens = moe.alloc_attn_workspace(0, n, Hkv, Hkv, D), ints(kv_lens)

    def call():
        return moe.kv_evict(kc, vc, table, lens, w, out_table, budget, first, last, *out, workspace=ws)
    got = call()
    assert all(a is b for a, b in zip(got, out))
    want, k, v = [x.clone() for x in out], kc.clone(), vc.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for x in out:
        x.fill_(5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(out, want))
    assert torch.equal(kc.view(torch.int16), k.view(torch.int16)) and torch.equal(vc.view(torch.int16), v.view(torch.int16))


# ------------------------------------------------------------ used together
def test_evict_then_decode():
    """A prompt served with a budget: its rows' weights, the eviction, and decode steps that append behind the kept keys
    and add to their weights, against attention over the kept keys."""
    g = gen_of(23)
    Hq, Hkv, D, page, n, steps, budget = 8, 2, 64, 16, [150, 40], 3, 64
    table = moe.rope_table(512, D)
    per = 12
    kc, vc = (torch.zeros(6 * per, Hkv, page, D, dtype=BF, device="cuda") for _ in range(2))
    pages = ints([list(range(per)), list(range(per, 2 * per))])
    spare = ints([list(range(2 * per, 3 * per)), list(range(3 * per, 4 * per))])

    def rows(T):
        return [rand(g, T, h, D) for h in (Hq, Hkv, Hkv)]
    q, k, v = rows(sum(n))
    slots = ints([int(pages[s, t // page]) * page + t % page for s in range(2) for t in range(n[s])])
    q = moe.rope_append(q, k, v, table, ints([t for x in n for t in range(x)]), slots, kc, vc)
    lse = torch.empty(sum(n), Hq, device="cuda")
    moe.attn_prefill_paged(q, kc, vc, pages, starts(n), ints(n), lse=lse)
    w = torch.zeros(2, Hkv, 256, device="cuda")
    moe.attn_key_weights(q, kc, pages, starts(n), ints(n), lse, w)
    want, tol = weights_reference(q, n, n, kc, pages, True, D ** -0.5, lse, torch.zeros_like(w))
    ref.check(w, want, tol, "weights")
    lens, new_w, kept = moe.kv_evict(kc, vc, pages, ints(n), w, spare, budget, keep_first=4, keep_last=16)
    assert lens.tolist() == [64, 40]
    held = []                                            # (keys, values) of each sequence and head that are left
    for s in range(2):
        ids = kept[s, :, :int(lens[s])].long()
        kk, vv = (ref.paged(c, pages[s], n[s]) for c in (kc, vc))
        held.append([torch.stack([x[h][ids[h]] for h in range(Hkv)]) for x in (kk, vv)])
    w = torch.nn.functional.pad(new_w, (0, 16)).contiguous()
    for i in range(steps):
        q, k, v = rows(2)
        slots = ints([int(spare[s, (int(lens[s])) // page]) * page + int(lens[s]) % page for s in range(2)])
        q = moe.rope_append(q, k, v, table, ints([x + i for x in n]), slots, kc, vc)
        for s in range(2):
            p, r = int(slots[s]) // page, int(slots[s]) % page
            held[s] = [torch.cat([x, c[p, :, r][:, None]], 1) for x, c in zip(held[s], (kc, vc))]
        lens = lens + 1
        lse = torch.empty(2, Hq, device="cuda")
        out = moe.attn_decode(q, kc, vc, spare, lens, lse=lse)
        before = w.clone()
        moe.attn_key_weights(q, kc, spare, ints([0, 1, 2]), lens, lse, w)
        want, tol = weights_reference(q, [1, 1], lens.tolist(), kc, spare, True, D ** -0.5, lse, before)
        ref.check(w, want, tol, "weights of a step")
        for s in range(2):
            o, le, to, tl = ref.attend(q[s:s + 1], held[s][0], held[s][1], D ** -0.5)
            ref.check(out[s:s + 1], o, to, "out")
            ref.check(lse[s:s + 1], le, tl, "lse")


@pytest.mark.parametrize("D,page,dtype", [(128, 16, BF), (64, 64, HF)])
def test_served_from_8_bits(D, page, dtype):
    """Prompts in chunks and decode steps over a cache in 8 bits, with positions of three axes and a prefix that the
    sequences share: each call against attention over what the cache then holds, and its new rows against their codes'
    bound."""
    g = gen_of(29)
    Hq, Hkv, B, shared = 8, 2, 3, 64
    table, axes = moe.rope_table(2048, D), moe.rope_axes(D, (D // 2 - D // 4, D // 8, D // 8), True)
    kc, vc, sc = moe.alloc_fp8_cache(4 + 40 * 16 // page, Hkv, page, D)
    free = list(range(kc.shape[0]))

    def take(tokens):
        got = [free.pop() for _ in range((tokens + page - 1) // page)]
        return got

    def append(T, pages, qs, lens):
        q, k, v = (rand(g, T, h, D, dtype=dtype) for h in (Hq, Hkv, Hkv))
        pos = torch.randint(0, 2048, (3, T), generator=g, device="cuda", dtype=torch.int32)
        out = moe.rope_append_fp8(q, k, v, table, pos, pages, ints(qs), ints(lens), kc, vc, sc, axes=axes)
        return out, v

    prefix = take(shared)
    pre = ints([prefix])
    q, v = append(shared, pre, [0, shared], [shared])
    got = c8.rows(vc, sc, 1, pre[0], shared)
    want = v.double().transpose(0, 1)
    ref.check(got, want, 2.0 ** -4 * want.abs() + 2.0 ** -9 * 2.0 ** -4, "values")
    own = [take(130) for _ in range(B)]
    pages = ints(own)
    both = ints([prefix + p for p in own])
    have = [0] * B
    for chunk in ([20, 1, 33], [50, 7, 0], [3, 60, 17]):
        T, qs = sum(chunk), [0, chunk[0], chunk[0] + chunk[1], sum(chunk)]
        have = [a + b for a, b in zip(have, chunk)]
        q, _ = append(T, pages, qs, have)
        lse = torch.empty(T, Hq, device="cuda")
        out = moe.attn_prefill_paged_fp8(q, kc, vc, sc, both, ints(qs), ints([shared + n for n in have]), lse=lse)
        for s in range(B):
            m = shared + have[s]
            k64, v64 = c8.rows(kc, sc, 0, both[s], m), c8.rows(vc, sc, 1, both[s], m)
            rows = slice(qs[s], qs[s + 1])
            o, le, to, tl = c8.attend(q[rows], k64, v64, D ** -0.5, ref.causal(chunk[s], m, q.device), parts=True)
            ref.check(out[rows], o, to, "prompt rows")
            ref.check(lse[rows], le, tl, "their log-sums")
    for _ in range(4):
        have = [n + 1 for n in have]
        q, _ = append(B, pages, list(range(B + 1)), have)
        out = moe.attn_decode_fp8(q, kc, vc, sc, pages, ints(have), pre[0].contiguous(), shared)
        for s in range(B):
            k64, v64 = (torch.cat([c8.rows(c, sc, x, pre[0], shared), c8.rows(c, sc, x, pages[s], have[s])], 1)
                        for x, c in ((0, kc), (1, vc)))
            o, le, to, tl = c8.attend(q[s:s + 1], k64, v64, D ** -0.5)
            ref.check(out[s:s + 1], o, to, "decode")


@pytest.mark.parametrize("wait", [2, 4, 5])
@pytest.mark.parametrize("D", [128, 64])
def test_key_weights_waits_that_give_up(wait, D):
    """Loads of keys and rows and the products of the tensor cores' kernel: a barrier that never completes ends the call
    with a report, and the next call on the workspace is right."""
    import test_gpu_attention_waits as waits
    q_lens, kv_lens, Hq, Hkv = [40, 60], [700, 900], 8, 2
    kc, _, table, _ = page_pool(kv_lens, 16, Hkv, D, BF, 35)
    q = rand(gen_of(36), 100, Hq, D)
    lse = torch.full((100, Hq), 5.0, device="cuda")
    ws = moe.alloc_attn_workspace(100, 2, Hq, Hkv, D)
    waits.times_out(lambda: moe.attn_key_weights(q, kc, table, starts(q_lens), ints(kv_lens), lse,
                                                 torch.zeros(2, Hkv, 900, device="cuda"), workspace=ws), ws, wait)


def test_offsets_beyond_32_bits():
    """The same calls with a sequence's pages at the start of a cache of more than 2^32 elements and at its end: the same
    bits."""
    Hq, Hkv, D, page, n = 16, 8, 128, 256, 700
    pages = (1 << 32) // (Hkv * page * D) + 12
    low, spare = ints([[1, 4, 2]]), ints([[6]])
    high, high_spare = low + (pages - 8), spare + (pages - 8)
    g = gen_of(41)
    table = moe.rope_table(1024, D)
    q, k, v = (rand(g, n, h, D) for h in (Hq, Hkv, Hkv))
    qs, lens, pos = ints([0, n]), ints([n]), torch.arange(n, dtype=torch.int32, device="cuda")
    k8, v8 = (torch.empty(pages, Hkv, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    sc = torch.empty(pages, Hkv, page // 16, 2, device="cuda")
    got = []
    for t in (low, high):
        x = moe.rope_append_fp8(q, k, v, table, pos, t, qs, lens, k8, v8, sc)
        ws = moe.alloc_attn_workspace(n, 1, Hq, Hkv, D)
        got.append([moe.attn_prefill_paged_fp8(x, k8, v8, sc, t, qs, lens, workspace=ws),
                    moe.attn_decode_fp8(x[-1:], k8, v8, sc, t, lens)])
        assert moe.read_status(ws) == 0 and not any(o.isnan().any() for o in got[-1])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    del k8, v8, sc
    kc, vc = (torch.empty(pages, Hkv, page, D, dtype=BF, device="cuda") for _ in range(2))
    got = []
    for t, to in ((low, spare), (high, high_spare)):
        slots = (t[0].long()[pos.long() // page] * page + pos.long() % page).to(torch.int32)
        x = moe.rope_append(q, k, v, table, pos, slots, kc, vc)
        lse = torch.empty(n, Hq, device="cuda")
        moe.attn_prefill_paged(x, kc, vc, t, qs, lens, lse=lse)
        many, few = torch.zeros(1, Hkv, n, device="cuda"), torch.zeros(1, Hkv, n, device="cuda")
        moe.attn_key_weights(x, kc, t, qs, lens, lse, many)
        moe.attn_key_weights(x[-3:], kc, t, ints([0, 3]), lens, lse[-3:], few)
        out = moe.kv_evict(kc, vc, t, lens, many, to, 200, 4, 30)
        got.append([many, few, *out, kc[int(to)].clone()[:, :200], vc[int(to)].clone()[:, :200]])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert bool((got[0][0] > 0).any()) and int(got[0][2]) == 200
