"""GPU tests of the attention operators against their definitions in 64 bits:
norms and rotary positions with the append to the paged cache, attention over
packed and paged prompts, and decode over the cache with a shared prefix."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_reference as ref  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
MOE_ERR_DEVICE = -5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


def rand(gen, *shape, dtype=BF, mul=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * mul).to(dtype)


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(lens):
    s = [0]
    for x in lens:
        s.append(s[-1] + x)
    return ints(s)


# ------------------------------------------------------------ rope_append
ROPE = [
    # T, Hq, Hkv, D, rot, interleaved, norm, page, dtype
    (1, 32, 4, 128, 128, False, True, 16, BF),
    (1, 1, 1, 64, 16, True, False, 16, HF),
    (5, 7, 1, 128, 64, False, True, 32, HF),
    (33, 6, 3, 64, 64, False, True, 64, BF),
    (33, 6, 3, 64, 32, True, True, 16, BF),
    (257, 8, 8, 128, 128, True, False, 128, BF),
    (130, 12, 2, 128, 32, False, False, 256, HF),
    (19, 4, 2, 64, 48, False, True, 16, BF),
    (19, 4, 2, 128, 0, False, True, 16, BF),
    (700, 32, 4, 128, 128, False, True, 16, BF),
]


def rope_case(T, Hq, Hkv, D, rot, interleaved, norm, page, dtype, seed=0):
    g = gen_of(seed)
    qkv = rand(g, T, (Hq + 2 * Hkv) * D + 8, dtype=dtype, mul=2.0)   # rows with 8 elements of padding
    q = qkv[:, :Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    v = qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(T, Hkv, D)
    pages = (T + page - 1) // page + 2
    table = moe.rope_table(5000, rot, base=10000.0) if rot else torch.zeros(5000, 0, device="cuda")
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    kc, vc = rand(g, pages, Hkv, page, D, dtype=dtype), rand(g, pages, Hkv, page, D, dtype=dtype)
    qn = 1 + 0.3 * torch.randn(D, generator=g, device="cuda") if norm else None
    kn = 1 + 0.3 * torch.randn(D, generator=g, device="cuda") if norm else None
    return q, k, v, table, pos, slots, kc, vc, qn, kn


def rope_check(q, k, v, table, pos, slots, kc0, vc0, kc, vc, qn, kn, rot, interleaved, out, eps=1e-6, skip=()):
    keep = torch.ones(q.shape[0], dtype=torch.bool)
    keep[list(skip)] = False
    rows = table[pos.long().clamp(0, table.shape[0] - 1)]
    cos, sin = rows[:, :rot // 2], rows[:, rot // 2:]
    want = ref.rope(q, qn, eps, cos, sin, rot, interleaved)[keep.cuda()]
    ref.check(out[keep.cuda()], want, ref.rope_bound(want, q.dtype), "q")
    page = kc.shape[2]
    wk = kc0.double().clone()
    tk = torch.zeros_like(wk)
    wv = vc0.clone()
    kk = ref.rope(k, kn, eps, cos, sin, rot, interleaved)
    for t in range(q.shape[0]):
        s = int(slots[t])
        if s < 0 or not keep[t]:
            continue
        wk[s // page, :, s % page] = kk[t]
        tk[s // page, :, s % page] = ref.rope_bound(kk[t], q.dtype)
        wv[s // page, :, s % page] = v[t]
    ref.check(kc, wk, tk, "k cache")            # rows that no token owns: unchanged, bound 0
    assert torch.equal(vc, wv)


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(map(str, c)))
def test_rope_append(case):
    T, Hq, Hkv, D, rot, inter, norm, page, dtype = case
    q, k, v, table, pos, slots, kc, vc, qn, kn = rope_case(*case)
    slots[T // 2] = -1 if T > 1 else slots[0]
    kc0, vc0 = kc.clone(), vc.clone()
    ws = moe.alloc_attn_workspace(T, 0, Hq, Hkv, D)
    out = moe.rope_append(q, k, v, table, pos, slots, kc, vc, qn, kn, interleaved=inter, workspace=ws)
    assert moe.read_status(ws) == 0
    rope_check(q, k, v, table, pos, slots, kc0, vc0, kc, vc, qn, kn, rot, inter, out)


def test_rope_append_in_place_and_zero_rows():
    T, Hq, Hkv, D = 40, 8, 2, 128
    q, k, v, table, pos, slots, kc, vc, qn, kn = rope_case(T, Hq, Hkv, D, 128, False, True, 16, BF, seed=3)
    q, k = q.contiguous(), k.contiguous()
    k[3] = 0                                   # a zero row: the norm divides by sqrt(eps)
    q[4] = 0
    kc0, vc0, q0 = kc.clone(), vc.clone(), q.clone()
    out = moe.rope_append(q, k, v, table, pos, slots, kc, vc, qn, kn, q_out=q)
    torch.cuda.synchronize()
    assert out is q
    rope_check(q0, k, v, table, pos, slots, kc0, vc0, kc, vc, qn, kn, 128, False, out)


def test_rope_append_reports_bad_indices():
    T, Hq, Hkv, D, page = 20, 4, 2, 64, 16
    q, k, v, table, pos, slots, kc, vc, qn, kn = rope_case(T, Hq, Hkv, D, 64, False, False, page, BF, seed=4)
    ws = moe.alloc_attn_workspace(T, 0, Hq, Hkv, D)
    for what in ("position", "negative position", "slot"):
        p, s = pos.clone(), slots.clone()
        kc1, vc1 = kc.clone(), vc.clone()
        if what == "position":
            p[7] = 5000
        elif what == "negative position":
            p[7] = -1
        else:
            s[7] = kc.shape[0] * page
        out = moe.rope_append(q, k, v, table, p, s, kc1, vc1, workspace=ws)
        assert moe.read_status(ws) == MOE_ERR_DEVICE
        rope_check(q, k, v, table, p, s, kc, vc, kc1, vc1, None, None, 64, False, out, skip=(7,))
    moe.rope_append(q, k, v, table, pos, slots, kc, vc, workspace=ws)
    assert moe.read_status(ws) == 0


# ------------------------------------------------------------ prefill
def packed_case(q_lens, kv_lens, Hq, Hkv, D, dtype, seed, strided=False, junk=False):
    """Packed q, k, v; with junk, NaN and infinities lie between and after
    the sequences' keys (kv_starts then skips none: junk only after the end)."""
    g = gen_of(seed)
    T, Tk = sum(q_lens), sum(kv_lens)
    pad = 8 if strided else 0
    q = rand(g, max(T, 1), Hq, D + pad, dtype=dtype, mul=2.5)[:T, :, :D]
    k = rand(g, Tk + 40, Hkv, D + pad, dtype=dtype)[..., :D]
    v = rand(g, Tk + 40, Hkv, D + pad, dtype=dtype)[..., :D]
    if junk:
        k[Tk:] = float("nan")
        v[Tk:] = float("inf")
    return q, k, v


def prefill_reference(q, q_lens, keys, causal, scale):
    """keys(s) -> (k, v) [Hkv, m, D] of sequence s."""
    outs = [[], [], [], []]
    at = 0
    for s, n in enumerate(q_lens):
        k, v = keys(s)
        seen = ref.causal(n, k.shape[1], q.device) if causal else None
        for o, x in zip(outs, ref.attend(q[at:at + n], k, v, scale, seen)):
            o.append(x)
        at += n
    return [torch.cat(o) for o in outs]


PREFILL = [
    # q_lens, kv_lens (None: the same), Hq, Hkv, D, causal, dtype, strided
    ([1], None, 8, 1, 128, True, BF, False),
    ([1, 1, 1], [1, 40, 130], 4, 4, 64, True, HF, False),
    ([127, 128, 129], None, 4, 2, 128, True, BF, True),
    ([0, 5, 0, 300, 0], None, 6, 2, 64, True, BF, False),
    ([33, 64, 257], None, 7, 1, 128, True, HF, True),
    ([33, 64, 257], None, 12, 12, 64, False, HF, False),
    ([100, 7, 9], [40, 0, 9], 8, 2, 128, True, BF, False),      # more rows than keys: rows that see none
    ([100, 7], [513, 0], 8, 2, 128, False, BF, False),
    ([17, 300], [1000, 700], 16, 1, 128, True, BF, False),
    ([5, 3], [300, 129], 128, 1, 64, True, BF, False),          # every head on one key-value head
    ([40, 65], None, 96, 3, 64, True, HF, False),
    ([1500], None, 4, 1, 128, True, BF, False),
    ([20] * 70, None, 4, 2, 64, True, BF, False),
    ([2, 700], [1, 900], 10, 2, 128, True, HF, False),
]


@pytest.mark.parametrize("case", PREFILL, ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}-{sum(c[0])}")
def test_prefill_packed(case):
    q_lens, kv_lens, Hq, Hkv, D, causal, dtype, strided = case
    kv_lens = q_lens if kv_lens is None else kv_lens
    q, k, v = packed_case(q_lens, kv_lens, Hq, Hkv, D, dtype, 11, strided, junk=True)
    at = [int(x) for x in starts(kv_lens)]
    lse = torch.full((q.shape[0], Hq), 7.0, device="cuda")
    ws = moe.alloc_attn_workspace(q.shape[0], len(q_lens), Hq, Hkv, D)
    out = moe.attn_prefill(q, k, v, starts(q_lens), starts(kv_lens), causal=causal, lse=lse, workspace=ws)
    assert moe.read_status(ws) == 0
    o, le, to, tl = prefill_reference(q, q_lens, lambda s: (k[at[s]:at[s + 1]].transpose(0, 1),
                                                            v[at[s]:at[s + 1]].transpose(0, 1)), causal, D ** -0.5)
    ref.check(out, o, to, "out")
    ref.check(lse, le, tl, "lse")


def page_pool(lens, page, Hkv, D, dtype, seed, extra_pages=0, spare=3):
    """A pool whose unused rows and pages hold NaN and infinities, page lists
    (their unused entries out of range), and each sequence's keys."""
    g = gen_of(seed)
    need = [(n + page - 1) // page for n in lens]
    pool = sum(need) + extra_pages + spare
    kc = torch.full((pool, Hkv, page, D), float("nan"), dtype=dtype, device="cuda")
    vc = torch.full((pool, Hkv, page, D), float("inf"), dtype=dtype, device="cuda")
    order = torch.randperm(pool, generator=g, device="cuda").tolist()
    table = torch.full((len(lens), max(max(need, default=0), 1) + 1), 1 << 30, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        for j in range(need[s]):
            rows = min(page, n - j * page)
            p = order[at]
            table[s, j] = p
            kc[p, :, :rows] = rand(g, Hkv, rows, D, dtype=dtype)
            vc[p, :, :rows] = rand(g, Hkv, rows, D, dtype=dtype)
            at += 1
    return kc, vc, table.cuda(), order[at:]


PAGED = [
    # q_lens, kv_lens, Hq, Hkv, D, causal, page, dtype
    ([1, 40, 130], [1, 200, 130], 8, 2, 128, True, 16, BF),
    ([64, 3], [1000, 515], 8, 1, 128, True, 32, BF),
    ([100], [777], 4, 4, 64, False, 64, HF),
    ([129, 0, 31], [129, 50, 1031], 7, 1, 64, True, 128, BF),
    ([50, 60], [300, 20], 6, 3, 128, True, 256, HF),
    ([1, 2, 3, 4], [3000, 0, 5, 4], 32, 4, 128, True, 16, BF),
    ([8], [9000], 8, 1, 128, True, 64, BF),
]


@pytest.mark.parametrize("case", PAGED, ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}-p{c[6]}-{sum(c[1])}")
def test_prefill_paged(case):
    q_lens, kv_lens, Hq, Hkv, D, causal, page, dtype = case
    kc, vc, table, _ = page_pool(kv_lens, page, Hkv, D, dtype, 21)
    q = rand(gen_of(22), sum(q_lens), Hq, D, dtype=dtype, mul=2.5)
    lse = torch.empty(q.shape[0], Hq, device="cuda")
    ws = moe.alloc_attn_workspace(q.shape[0], len(q_lens), Hq, Hkv, D)
    out = moe.attn_prefill_paged(q, kc, vc, table, starts(q_lens), ints(kv_lens), causal=causal, lse=lse, workspace=ws)
    assert moe.read_status(ws) == 0

    def keys(s):
        pages = table[s, :(kv_lens[s] + page - 1) // page]
        return ref.paged(kc, pages, kv_lens[s]), ref.paged(vc, pages, kv_lens[s])
    o, le, to, tl = prefill_reference(q, q_lens, keys, causal, D ** -0.5)
    ref.check(out, o, to, "out")
    ref.check(lse, le, tl, "lse")


# A few sequences of thousands of keys: chunks of long prompts, short sequences
# among long ones, rows without keys, keys split over blocks or not
LONG = [
    # q_lens, kv_lens, Hq, Hkv, D, causal, page, dtype
    ([300, 17, 1, 512], [4100, 3500, 4000, 512], 32, 4, 128, True, 16, BF),
    ([1400], [5001], 16, 8, 64, True, 64, HF),
    ([200, 0, 90, 64], [4000, 100, 0, 64], 16, 16, 64, False, 32, HF),
    ([150, 400], [60, 3500], 48, 4, 128, True, 128, BF),
    ([1] * 70 + [40], [5] * 70 + [5000], 8, 2, 128, True, 16, BF),
    ([129, 1200], [9000, 1200], 8, 4, 128, False, 256, BF),
]


@pytest.mark.parametrize("paged", [True, False], ids=["paged", "packed"])
@pytest.mark.parametrize("case", LONG, ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}-{sum(c[0])}-{max(c[1])}")
def test_prefill_long(case, paged):
    q_lens, kv_lens, Hq, Hkv, D, causal, page, dtype = case
    q = rand(gen_of(22), sum(q_lens), Hq, D, dtype=dtype, mul=2.5)
    lse = torch.full((q.shape[0], Hq), 7.0, device="cuda")
    ws = moe.alloc_attn_workspace(q.shape[0], len(q_lens), Hq, Hkv, D)
    if paged:
        kc, vc, table, _ = page_pool(kv_lens, page, Hkv, D, dtype, 21)

        def call(lse):
            return moe.attn_prefill_paged(q, kc, vc, table, starts(q_lens), ints(kv_lens), causal=causal, lse=lse,
                                          workspace=ws)

        def keys(s):
            pages = table[s, :(kv_lens[s] + page - 1) // page]
            return ref.paged(kc, pages, kv_lens[s]), ref.paged(vc, pages, kv_lens[s])
    else:
        _, k, v = packed_case(q_lens, kv_lens, Hq, Hkv, D, dtype, 23, junk=True)
        at = [int(x) for x in starts(kv_lens)]

        def call(lse):
            return moe.attn_prefill(q, k, v, starts(q_lens), starts(kv_lens), causal=causal, lse=lse, workspace=ws)

        def keys(s):
            return k[at[s]:at[s + 1]].transpose(0, 1), v[at[s]:at[s + 1]].transpose(0, 1)
    out = call(lse)
    assert moe.read_status(ws) == 0
    o, le, to, tl = prefill_reference(q, q_lens, keys, causal, D ** -0.5)
    ref.check(out, o, to, "out")
    ref.check(lse, le, tl, "lse")
    assert torch.equal(out, call(lse))


def test_prefill_long_reports_bad_lengths_and_pages():
    q_lens, kv_lens, Hq, Hkv, D, page = [300, 17, 1, 512], [4100, 3500, 4000, 512], 32, 4, 128, 16
    kc, vc, table, _ = page_pool(kv_lens, page, Hkv, D, BF, 21)
    q = rand(gen_of(22), sum(q_lens), Hq, D, mul=2.5)
    ws = moe.alloc_attn_workspace(q.shape[0], 4, Hq, Hkv, D)

    def call(table, kv):
        out = moe.attn_prefill_paged(q, kc, vc, table, starts(q_lens), ints(kv), workspace=ws)
        return out, moe.read_status(ws)
    clean, status = call(table, kv_lens)
    assert status == 0
    out, status = call(table, [4100, 1 << 30, 4000, 512])     # the second counts as empty
    assert status != 0
    rest = list(range(300)) + list(range(317, sum(q_lens)))
    # (the other sequences' keys may be split in other places: a rounding of the type, twice on each side)
    assert bool((out[300:317] == 0).all())
    assert float((out[rest].float() - clean[rest].float()).abs().max()) <= 4 * 2.0 ** -8 * float(clean[rest].float().abs().max())
    bad = table.clone()
    bad[2, 7] = 1 << 29
    assert call(bad, kv_lens)[1] != 0
    again, status = call(table, kv_lens)
    assert status == 0 and torch.equal(again, clean)


def test_prefill_scales_and_extreme_logits():
    # scale 0 (every key alike), a negative scale, and logits far apart
    q, k, v = packed_case([200], [200], 4, 2, 128, BF, 31)
    q[50:60] *= 40
    for scale in (0.0, -0.05, 0.3):
        lse = torch.empty(200, 4, device="cuda")
        out = moe.attn_prefill(q, k, v, starts([200]), starts([200]), scale=scale, lse=lse)
        o, le, to, tl = prefill_reference(q, [200], lambda s: (k[:200].transpose(0, 1), v[:200].transpose(0, 1)),
                                          True, scale)
        ref.check(out, o, to, f"out, scale {scale}")
        ref.check(lse, le, tl, f"lse, scale {scale}")


def test_prefill_growing_logits():
    # each key block's logits exceed the ones before it: the running maximum moves all the way
    n, D = 1200, 128
    q, k, v = packed_case([64], [n], 4, 1, D, BF, 32)
    k[:n] = k[:n] * torch.linspace(0.1, 3.0, n, device="cuda")[:, None, None].to(BF)
    q[:] = q.abs()
    k[:n] = k[:n].abs()
    out = moe.attn_prefill(q, k, v, starts([64]), starts([n]), causal=False)
    o, _, to, _ = prefill_reference(q, [64], lambda s: (k[:n].transpose(0, 1), v[:n].transpose(0, 1)), False, D ** -0.5)
    ref.check(out, o, to, "out")


def test_prefill_neighbours_do_not_leak():
    # a sequence of NaN and infinities beside finite ones
    lens = [70, 50, 90]
    q, k, v = packed_case(lens, lens, 4, 2, 64, BF, 33)
    clean = moe.attn_prefill(q, k, v, starts(lens), starts(lens))
    k[70:120] = float("nan")
    v[70:120] = float("inf")
    out = moe.attn_prefill(q, k, v, starts(lens), starts(lens))
    assert torch.equal(out[:70], clean[:70]) and torch.equal(out[120:], clean[120:])


def test_prefill_same_bits_twice_and_alone():
    # the result of a sequence does not change from run to run
    lens = [300, 900, 17]
    q, k, v = packed_case(lens, lens, 8, 2, 128, BF, 34)
    a = moe.attn_prefill(q, k, v, starts(lens), starts(lens))
    b = moe.attn_prefill(q, k, v, starts(lens), starts(lens))
    assert torch.equal(a, b)


# ------------------------------------------------------------ decode
DECODE = [
    # kv_lens, prefix, Hq, Hkv, D, page, dtype
    ([1], 0, 32, 4, 128, 16, BF),
    ([0], 0, 8, 2, 64, 16, BF),
    ([15, 16, 17, 0, 33], 0, 8, 2, 128, 16, BF),
    ([100, 700, 3], 0, 16, 2, 64, 32, HF),
    ([5000], 0, 32, 4, 128, 64, BF),
    ([20011, 7], 0, 8, 1, 128, 16, HF),
    ([64, 128, 129, 255], 0, 7, 1, 128, 128, BF),
    ([300, 40], 0, 48, 2, 128, 256, BF),                       # 24 heads share a key-value head
    ([130, 1, 77], 0, 128, 1, 64, 16, BF),                      # 128 of them
    ([12] * 300, 0, 2, 1, 64, 16, BF),
    ([10, 0, 300, 129], 1, 8, 2, 128, 16, BF),
    ([10, 0, 300, 129], 1000, 8, 2, 128, 16, BF),
    ([0, 0], 300, 4, 4, 64, 64, HF),
    ([33] * 70, 4097, 32, 4, 128, 16, BF),
    ([500, 2, 90], 20000, 6, 1, 128, 128, HF),
    ([17], 513, 128, 1, 64, 32, BF),
]


def decode_case(kv_lens, prefix, Hq, Hkv, D, page, dtype, seed=41):
    npre = (prefix + page - 1) // page
    kc, vc, table, free = page_pool(kv_lens, page, Hkv, D, dtype, seed, extra_pages=npre)
    g = gen_of(seed + 1)
    pre = ints(free[:npre]) if npre else None
    for j in range(npre):
        rows = min(page, prefix - j * page)
        kc[free[j], :, :rows] = rand(g, Hkv, rows, D, dtype=dtype)
        vc[free[j], :, :rows] = rand(g, Hkv, rows, D, dtype=dtype)
    q = rand(g, len(kv_lens), Hq, D, dtype=dtype, mul=2.5)
    return q, kc, vc, table, pre


def decode_reference(q, kc, vc, table, pre, kv_lens, prefix, page, scale):
    outs = [[], [], [], []]
    for b, n in enumerate(kv_lens):
        pages = table[b, :(n + page - 1) // page]
        k, v = ref.paged(kc, pages, n), ref.paged(vc, pages, n)
        if prefix:
            k = torch.cat([ref.paged(kc, pre, prefix), k], dim=1)
            v = torch.cat([ref.paged(vc, pre, prefix), v], dim=1)
        for o, x in zip(outs, ref.attend(q[b:b + 1], k, v, scale)):
            o.append(x)
    return [torch.cat(o) for o in outs]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}-B{len(c[0])}-{max(c[0])}-pre{c[1]}")
def test_decode(case):
    kv_lens, prefix, Hq, Hkv, D, page, dtype = case
    q, kc, vc, table, pre = decode_case(*case)
    lse = torch.full((len(kv_lens), Hq), 7.0, device="cuda")
    ws = moe.alloc_attn_workspace(len(kv_lens), len(kv_lens), Hq, Hkv, D)
    out = moe.attn_decode(q, kc, vc, table, ints(kv_lens), pre, prefix, lse=lse, workspace=ws)
    assert moe.read_status(ws) == 0
    o, le, to, tl = decode_reference(q, kc, vc, table, pre, kv_lens, prefix, page, D ** -0.5)
    ref.check(out, o, to, "out")
    ref.check(lse, le, tl, "lse")
    again = moe.attn_decode(q, kc, vc, table, ints(kv_lens), pre, prefix, workspace=ws)
    assert torch.equal(out, again)


# More keys of the rows' own than fit beside the prefix's kernel (the rest comes
# after it), more sequences than a block holds lengths of, and both
DECODE_MANY = [
    ([1500 + 37 * i for i in range(32)], 256, 8, 4, 64, 16, BF),
    ([0, 60000, 1, 4000, 40000], 700, 16, 2, 128, 64, HF),
    ([130 + i % 3 for i in range(400)], 2000, 32, 4, 128, 16, BF),
    ([90 + i % 50 for i in range(700)], 0, 8, 2, 64, 16, HF),
    ([0] * 280 + [3] * 20 + [5000], 64, 12, 1, 128, 32, BF),
]


@pytest.mark.parametrize("case", DECODE_MANY, ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}-B{len(c[0])}-{max(c[0])}-pre{c[1]}")
def test_decode_many_keys(case):
    test_decode(case)


@pytest.mark.parametrize("kv_lens,prefix", [([40], 0), ([9000], 0), ([300, 0, 5000], 512), ([0, 17], 4096)])
def test_decode_nan_query_stays_in_its_head(kv_lens, prefix):
    # a NaN that a row does see is in its result, whether the row's keys are in
    # one piece or joined from parts, and in no other head's
    q, kc, vc, table, pre = decode_case(kv_lens, prefix, 16, 2, 128, 16, BF)
    q[:, 5, 3] = float("nan")
    lse = torch.empty(len(kv_lens), 16, device="cuda")
    out = moe.attn_decode(q, kc, vc, table, ints(kv_lens), pre, prefix, lse=lse)
    sees = torch.tensor([n + prefix > 0 for n in kv_lens], device="cuda")
    assert bool(out[sees, 5].isnan().all()) and bool(lse[sees, 5].isnan().all())
    others = [h for h in range(16) if h != 5]
    assert not bool(out[:, others].isnan().any()) and not bool(lse[:, others].isnan().any())


def test_decode_strided_rows_and_scale():
    q, kc, vc, table, _ = decode_case([90, 200], 0, 8, 2, 64, 16, BF)
    wide = torch.zeros(2, 8 * 64 + 72, dtype=BF, device="cuda")
    wide[:, :512] = q.view(2, 512)
    rows = wide[:, :512].view(2, 8, 64)
    out = moe.attn_decode(rows, kc, vc, table, ints([90, 200]), scale=0.3)
    o, _, to, _ = decode_reference(q, kc, vc, table, None, [90, 200], 0, 16, 0.3)
    ref.check(out, o, to, "out")


def test_offsets_past_32_bits():
    # a cache of more than 2^31 elements (and 2^32 bytes) for each of k and v
    page, Hkv, D = 256, 8, 128
    pool = (1 << 31) // (page * Hkv * D) + 3
    kc = torch.empty(pool, Hkv, page, D, dtype=BF, device="cuda")
    vc = torch.empty(pool, Hkv, page, D, dtype=BF, device="cuda")
    g = gen_of(51)
    ids = [pool - 1, 0, pool - 2]
    T, Hq = 300, 16
    k, v, q = rand(g, T, Hkv, D), rand(g, T, Hkv, D), rand(g, T, Hq, D)
    slots = ints([ids[t // page] * page + t % page for t in range(T)])
    table = moe.rope_table(400, 128)
    out = moe.rope_append(q, k, v, table, ints(list(range(T))), slots, kc, vc)
    rows = table[:T]
    kk = ref.rope(k, None, 1e-6, rows[:, :64], rows[:, 64:], 128, False)
    got = ref.paged(kc, ints(ids[:2]), T).transpose(0, 1)
    ref.check(got, kk, ref.rope_bound(kk, BF), "k cache")
    assert torch.equal(ref.paged(vc, ints(ids[:2]), T).transpose(0, 1), v)
    lists = ints([ids])
    K, V = ref.paged(kc, ints(ids[:2]), T), ref.paged(vc, ints(ids[:2]), T)
    res = moe.attn_prefill_paged(out, kc, vc, lists, starts([T]), ints([T]))
    o, _, to, _ = prefill_reference(out, [T], lambda s: (K, V), True, D ** -0.5)
    ref.check(res, o, to, "prefill")
    one = moe.attn_decode(out[-1:], kc, vc, lists, ints([T]))
    o, _, to, _ = ref.attend(out[-1:], K, V, D ** -0.5)
    ref.check(one, o, to, "decode")


# ------------------------------------------------------------ errors, streams, graphs
def test_attention_reports_bad_indices():
    page, Hq, Hkv, D = 16, 4, 2, 64
    lens = [40, 90, 20]
    q, kc, vc, table, _ = decode_case(lens, 0, Hq, Hkv, D, page, BF)
    ws = moe.alloc_attn_workspace(400, 8, Hq, Hkv, D)
    moe.attn_decode(q, kc, vc, table, ints(lens), workspace=ws)
    assert moe.read_status(ws) == 0
    want, _, tol, _ = decode_reference(q, kc, vc, table, None, lens, 0, page, D ** -0.5)

    def others(out):                       # the sequences beside the bad one are right
        for b in (0, 2):
            ref.check(out[b], want[b], tol[b], f"sequence {b}")
    for bad in (-1, kc.shape[0]):
        t = table.clone()
        t[1, 2] = bad
        out = moe.attn_decode(q, kc, vc, t, ints(lens), workspace=ws)
        assert moe.read_status(ws) == MOE_ERR_DEVICE
        others(out)
    for n in (-1, table.shape[1] * page + 1):
        out = moe.attn_decode(q, kc, vc, table, ints([40, n, 20]), workspace=ws)
        assert moe.read_status(ws) == MOE_ERR_DEVICE
        others(out)
    pre = ints([kc.shape[0], 0])
    moe.attn_decode(q, kc, vc, table, ints(lens), pre, 20, workspace=ws)
    assert moe.read_status(ws) == MOE_ERR_DEVICE
    moe.attn_decode(q, kc, vc, table, ints(lens), workspace=ws)
    assert moe.read_status(ws) == 0

    rows = rand(gen_of(5), 130, Hq, D)
    t = table.clone()
    t[2, 1] = -5
    moe.attn_prefill_paged(rows, kc, vc, t, starts([30, 80, 20]), ints(lens), workspace=ws)
    assert moe.read_status(ws) == MOE_ERR_DEVICE
    k = rand(gen_of(6), 130, Hkv, D)
    for qs, ks in (([0, 30, 200, 130], [0, 30, 110, 130]),       # past the rows
                   ([0, 30, 110, 130], [0, 30, 110, 131]),       # past the keys
                   ([0, 30, 110, 130], [0, 50, 20, 130]),        # not ascending
                   ([0, 30, 110, 130], [0, -7, 110, 130])):
        moe.attn_prefill(rows, k, k, ints(qs), ints(ks), workspace=ws)
        assert moe.read_status(ws) == MOE_ERR_DEVICE, (qs, ks)
    moe.attn_prefill(rows, k, k, starts([30, 80, 20]), starts([30, 80, 20]), workspace=ws)
    assert moe.read_status(ws) == 0


def test_other_streams_and_graph_replay():
    lens = [200, 45, 800, 1]
    q, kc, vc, table, pre = decode_case(lens, 100, 8, 2, 128, 16, BF)
    n = ints(lens)
    rows, k, v = packed_case([300, 20], [300, 20], 8, 2, 128, BF, 61)
    qs = starts([300, 20])
    ws, ws2 = moe.alloc_attn_workspace(4, 4, 8, 2, 128), moe.alloc_attn_workspace(320, 2, 8, 2, 128)
    want_d = moe.attn_decode(q, kc, vc, table, n, pre, 100)
    want_p = moe.attn_prefill(rows, k, v, qs, qs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got_d = moe.attn_decode(q, kc, vc, table, n, pre, 100, stream=side)
    got_p = moe.attn_prefill(rows, k, v, qs, qs, stream=side)
    side.synchronize()
    assert torch.equal(got_d, want_d) and torch.equal(got_p, want_p)
    out_d, out_p = torch.empty_like(want_d), torch.empty_like(want_p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.attn_decode(q, kc, vc, table, n, pre, 100, out=out_d, workspace=ws)
        moe.attn_prefill(rows, k, v, qs, qs, out=out_p, workspace=ws2)
    for _ in range(3):
        out_d.zero_()
        out_p.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out_d, want_d) and torch.equal(out_p, want_p)
    # the replayed graph reads the lengths of the moment
    n.copy_(ints([10, 45, 3, 0]))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out_d, moe.attn_decode(q, kc, vc, table, n, pre, 100))


def test_empty_batches():
    kc = torch.zeros(2, 2, 16, 64, dtype=BF, device="cuda")
    none = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    kv = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    table = moe.rope_table(8, 64)
    assert moe.rope_append(none, kv, kv, table, e, e, kc, kc.clone()).shape == (0, 4, 64)
    assert moe.attn_prefill(none, kv, kv, starts([0, 0]), starts([0, 0])).shape == (0, 4, 64)
    assert moe.attn_decode(none, kc, kc.clone(), torch.empty(0, 3, dtype=torch.int32, device="cuda"), e).shape == (0, 4, 64)
    # rows, but no key at all
    q = torch.ones(3, 4, 64, dtype=BF, device="cuda")
    lse = torch.zeros(3, 4, device="cuda")
    out = moe.attn_prefill(q, kv, kv, starts([3]), starts([0]), lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
