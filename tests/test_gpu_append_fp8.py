"""GPU tests of rotary positions with several axes and of the append to a
paged cache in 8 bits, against their definitions in 64 bits."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_reference as ref  # noqa: E402
import cache8_reference as c8  # noqa: E402
from test_gpu_attention import BF, HF, gen_of, ints, rand, starts  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu

MOE_ERR_DEVICE = -5
MAX_POS = 700


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


def angles(table, positions, axes, rot):
    """cos, sin [T, rot / 2] of every token's pairs."""
    half = rot // 2
    if axes is None:
        got = table[positions.long()]
        return got[:, :half], got[:, half:]
    pair = torch.arange(half, device="cuda")
    at = positions.long()[axes.long()].T
    return table[at, pair], table[at, pair + half]


def projection(g, T, Hq, Hkv, D, dtype):
    qkv = rand(g, T, (Hq + 2 * Hkv) * D + 8, dtype=dtype, mul=2.0)     # rows with 8 elements of padding
    return (qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
            qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(T, Hkv, D))


def norms(g, D, on):
    return [1 + 0.3 * torch.randn(D, generator=g, device="cuda") if on else None for _ in range(2)]


# ------------------------------------------------------------ several axes
AXES = [
    # T, Hq, Hkv, D, rot, sections, in turns, interleaved, norm, dtype
    (1, 32, 4, 128, 128, (16, 24, 24), False, False, True, BF),
    (33, 6, 3, 64, 64, (12, 10, 10), True, True, False, HF),
    (257, 8, 8, 128, 64, (16, 16), False, False, True, BF),
    (130, 12, 2, 64, 48, (6, 6, 6, 6), True, False, False, HF),
    (19, 4, 2, 128, 32, (0, 16), False, True, True, BF),
    (1200, 32, 4, 128, 128, (44, 10, 10), True, False, True, BF),     # several heads to a group of lanes
    (5, 4, 2, 64, 64, (32,), False, False, False, BF),
]


def axes_case(case, seed=5):
    T, Hq, Hkv, D, rot, sections, turns, inter, norm, dtype = case
    g = gen_of(seed)
    q, k, v = projection(g, T, Hq, Hkv, D, dtype)
    table = moe.rope_table(MAX_POS, rot)
    pos = torch.randint(0, MAX_POS, (len(sections), T), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm((T // 16 + 2) * 16, generator=g, device="cuda")[:T].to(torch.int32)
    kc, vc = (rand(g, T // 16 + 2, Hkv, 16, D, dtype=dtype) for _ in range(2))
    return q, k, v, table, pos, slots, kc, vc, norms(g, D, norm), moe.rope_axes(rot, sections, turns)


@pytest.mark.parametrize("case", AXES, ids=lambda c: "-".join(map(str, c[:5])) + f"-{len(c[5])}axes")
def test_rope_append_axes(case):
    T, Hq, Hkv, D, rot, sections, turns, inter, norm, dtype = case
    q, k, v, table, pos, slots, kc, vc, (qn, kn), axes = axes_case(case)
    assert [int((axes == x).sum()) for x in range(len(sections))] == list(sections)
    kc0, vc0 = kc.clone(), vc.clone()
    ws = moe.alloc_attn_workspace(T, 0, Hq, Hkv, D)
    out = moe.rope_append(q, k, v, table, pos, slots, kc, vc, qn, kn, interleaved=inter, workspace=ws, axes=axes)
    assert moe.read_status(ws) == 0
    cos, sin = angles(table, pos, axes, rot)
    want = ref.rope(q, qn, 1e-6, cos, sin, rot, inter)
    ref.check(out, want, ref.rope_bound(want, dtype), "q")
    kk = ref.rope(k, kn, 1e-6, cos, sin, rot, inter)
    at = slots.long()
    ref.check(kc[at // 16, :, at % 16], kk, ref.rope_bound(kk, dtype), "k")
    assert torch.equal(vc[at // 16, :, at % 16], v)
    kc[at // 16, :, at % 16] = kc0[at // 16, :, at % 16]
    vc[at // 16, :, at % 16] = vc0[at // 16, :, at % 16]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)             # nothing else was written


def test_equal_positions_are_one_position():
    q, k, v, table, pos, slots, kc, vc, (qn, kn), axes = axes_case(AXES[0])
    pos[1:] = pos[0]
    kc1, vc1 = kc.clone(), vc.clone()
    a = moe.rope_append(q, k, v, table, pos, slots, kc, vc, qn, kn, axes=axes)
    b = moe.rope_append(q, k, v, table, pos[0].contiguous(), slots, kc1, vc1, qn, kn)
    assert torch.equal(a, b) and torch.equal(kc, kc1) and torch.equal(vc, vc1)


def test_axes_out_of_range_are_reported():
    case = AXES[1]
    q, k, v, table, pos, slots, kc, vc, (qn, kn), axes = axes_case(case)
    ws = moe.alloc_attn_workspace(case[0], 0, case[1], case[2], case[3])

    def status(pos, axes):
        moe.rope_append(q, k, v, table, pos, slots, kc, vc, qn, kn, workspace=ws, axes=axes)
        return moe.read_status(ws)
    assert status(pos, axes) == 0
    for bad in (3, 255):
        a = axes.clone()
        a[7] = bad
        assert status(pos, a) == MOE_ERR_DEVICE
    for bad in (-1, MAX_POS, 1 << 30):
        p = pos.clone()
        p[2, 5] = bad
        assert status(p, axes) == MOE_ERR_DEVICE


# ------------------------------------------------------------ append in 8 bits
APPEND = [
    # tokens before, new tokens, Hq, Hkv, D, rot, interleaved, norm, axes, page, dtype
    ([0], [1], 32, 4, 128, 128, False, True, 1, 16, BF),
    ([5, 15, 16, 31, 0], [1, 1, 1, 1, 1], 8, 2, 64, 32, True, False, 1, 16, HF),          # one token each
    ([5, 7], [2, 3], 8, 8, 128, 64, False, True, 3, 32, BF),
    ([0, 10, 0, 3, 100], [0, 40, 0, 0, 17], 6, 3, 64, 64, False, False, 2, 64, BF),       # sequences without tokens
    ([0], [300], 4, 1, 128, 128, True, True, 1, 128, HF),
    ([17, 0, 250], [33, 129, 6], 12, 2, 128, 0, False, True, 1, 256, BF),                 # no rotation
    ([1] * 70, [1] * 70, 4, 2, 64, 48, False, True, 4, 16, BF),                           # more sequences than 32
    ([3] * 40, [0, 2] * 20, 4, 2, 64, 16, False, False, 1, 16, HF),                       # as many tokens as sequences
    ([40, 0], [2000, 700], 32, 4, 128, 128, False, True, 1, 16, BF),                      # several heads to a group
    ([31], [1], 1, 1, 128, 128, False, False, 1, 16, BF),
]


def append_case(case, seed=9):
    before, new, Hq, Hkv, D, rot, inter, norm, n_axes, page, dtype = case
    g = gen_of(seed)
    T = sum(new)
    q, k, v = projection(g, T, Hq, Hkv, D, dtype)
    # tokens of very different sizes, so that scales of blocks differ and have to grow
    size = torch.exp2(3 * torch.randn(T, 1, 1, generator=g, device="cuda")).to(dtype)
    v = v * size
    if not norm:
        k = k * size
    table = moe.rope_table(MAX_POS, rot) if rot else torch.zeros(MAX_POS, 0, device="cuda")
    axes = None if n_axes == 1 else moe.rope_axes(rot, [rot // 2 - 2 * (n_axes - 1)] + [2] * (n_axes - 1), True)
    pos = torch.randint(0, MAX_POS, (T,) if n_axes == 1 else (n_axes, T), generator=g, device="cuda", dtype=torch.int32)
    need = [(b + n + page - 1) // page for b, n in zip(before, new)]
    pool = sum(need) + 2
    order = torch.randperm(pool, generator=g, device="cuda").tolist()
    table_pages = torch.full((len(new), max(max(need), 1) + 1), 1 << 30, dtype=torch.int32)     # unused entries out of range
    at = 0
    for s, n in enumerate(need):
        table_pages[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    kc, vc, scales = moe.alloc_fp8_cache(pool, Hkv, page, D)
    for c in (kc, vc):                                               # any bits, NaN among them
        c.view(torch.uint8).copy_(torch.randint(0, 256, c.shape, generator=g, device="cuda", dtype=torch.uint8))
    scales.copy_(torch.exp2(torch.randint(-12, 3, scales.shape, generator=g, device="cuda").float()))
    lens = ints([b + n for b, n in zip(before, new)])
    return q, k, v, table, pos, table_pages.cuda(), starts(new), lens, kc, vc, scales, norms(g, D, norm), axes


def check_append(case, q, k, v, table, pos, pages, kc0, vc0, sc0, kc, vc, sc, qn, kn, axes, out, skip=()):
    before, new, Hq, Hkv, D, rot, inter, norm, n_axes, page, dtype = case
    cos, sin = angles(table, pos, axes, rot)
    want = ref.rope(q, qn, 1e-6, cos, sin, rot, inter)
    ref.check(out, want, ref.rope_bound(want, dtype), "q")
    kk = ref.rope(k, kn, 1e-6, cos, sin, rot, inter)
    # fp32 before the rounding to a code: what rope_bound has without the rounding to the type
    off = 20 * 2.0 ** -24 * 1.5 * kk.abs().amax(-1, keepdim=True)
    kk, off, vv = kk.cpu(), off.cpu(), v.double().cpu()
    pages = pages.cpu()
    got = [c8.values(kc), c8.values(vc)]
    old = [c8.values(kc0), c8.values(vc0)]
    bits, bits0 = ([c.view(torch.uint8).cpu().clone() for c in cs] for cs in ((kc, vc), (kc0, vc0)))
    sc, sc0 = sc.cpu(), sc0.cpu()
    written = torch.zeros_like(sc, dtype=torch.bool)
    t = 0
    for s, (b, n) in enumerate(zip(before, new)):
        at = b
        while at < b + n:
            to = min(b + n, at // 16 * 16 + 16)
            p, r0 = int(pages[s, at // page]), at % page
            first, r1 = r0 // 16 * 16, r0 + to - at
            if s in skip:
                t, at = t + to - at, to
                continue
            for x, rows in enumerate((kk[t:t + to - at], vv[t:t + to - at])):
                for h in range(Hkv):
                    y = rows[:, h]
                    slack = off[t:t + to - at, h] if x == 0 else torch.zeros(1, 1, dtype=torch.float64)
                    fit = [c8.scale_of(float((y.abs() + d * slack).nan_to_num(0.0).clamp(min=0.0).max())) for d in (-1, 1)]
                    if r0 > first:
                        fit = [max(f, float(sc0[p, h, first // 16, x])) for f in fit]
                    e = float(sc[p, h, first // 16, x])
                    written[p, h, first // 16, x] = True
                    assert e in fit, (s, at, h, x, e, fit)
                    code = got[x][p, h, r0:r1]
                    if x == 1:
                        w = c8.round8(y / e)
                        assert torch.equal(code.nan_to_num(1e9), w.nan_to_num(1e9)), (s, at, h)
                    else:
                        # half a step: 2^-4 of a value, half of 2^-9 below the normal codes
                        ref.check(code * e, y, slack + 2.0 ** -4 * y.abs() + 2.0 ** -10 * e, "k codes")
                    if r0 > first:
                        w = c8.round8(old[x][p, h, first:r0] * (float(sc0[p, h, first // 16, x]) / e))
                        assert torch.equal(got[x][p, h, first:r0].nan_to_num(1e9), w.nan_to_num(1e9)), (s, at, h, "before")
                bits[x][p, :, first:r1] = bits0[x][p, :, first:r1]
            t, at = t + to - at, to
    assert torch.equal(sc[~written], sc0[~written])
    assert all(torch.equal(a, b) for a, b in zip(bits, bits0))           # nothing else was written


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}-{len(c[0])}seq-{sum(c[1])}tok-p{c[9]}")
def test_append(case):
    q, k, v, table, pos, pages, qs, lens, kc, vc, sc, (qn, kn), axes = append_case(case)
    kc0, vc0, sc0 = kc.clone(), vc.clone(), sc.clone()
    ws = moe.alloc_attn_workspace(q.shape[0], len(case[0]), case[2], case[3], case[4])
    out = moe.rope_append_fp8(q, k, v, table, pos, pages, qs, lens, kc, vc, sc, qn, kn, interleaved=case[6], axes=axes,
                              workspace=ws)
    assert moe.read_status(ws) == 0
    check_append(case, q, k, v, table, pos, pages, kc0, vc0, sc0, kc, vc, sc, qn, kn, axes, out)
    # the same again: scales that fit stay, codes too
    kc1, vc1, sc1 = kc.clone(), vc.clone(), sc.clone()
    moe.rope_append_fp8(q, k, v, table, pos, pages, qs, lens, kc, vc, sc, qn, kn, interleaved=case[6], axes=axes,
                        workspace=ws)
    for a, b in ((kc, kc1), (vc, vc1)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(sc, sc1)


def test_queries_are_those_of_the_16_bit_append():
    case = APPEND[2]
    q, k, v, table, pos, pages, qs, lens, kc, vc, sc, (qn, kn), axes = append_case(case)
    k16, v16 = (torch.zeros(2, case[3], 16, case[4], dtype=BF, device="cuda") for _ in range(2))
    a = moe.rope_append(q, k, v, table, pos, ints(list(range(5))), k16, v16, qn, kn, axes=axes)
    b = moe.rope_append_fp8(q, k, v, table, pos, pages, qs, lens, kc, vc, sc, qn, kn, axes=axes)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_values_that_are_not_ordinary(dtype):
    """Zeros, values beyond 57344, infinities, NaN, the smallest, exact ties between codes, block maxima of 448 times a power."""
    Hkv, D = 1, 64
    rows = torch.ones(64, D)
    rows[0:16] = 0
    rows[16, 3], rows[17, 4], rows[18, 5] = 60000, -65504, 1
    rows[32, 0], rows[33, 1], rows[34, 2] = float("inf"), -float("inf"), float("nan")
    rows[48:64] = 2.0 ** -20 if dtype == HF else 2.0 ** -30
    more = torch.zeros(64, D)
    more[0:16] = torch.arange(D) / 16 + 17 / 16            # around ties: steps of 1/8, 1/4 between codes
    more[16] = 448
    more[32] = 448.5 if dtype == HF else 450
    more[48] = 448 * 2.0 ** -9
    v = torch.cat([rows, more]).to(dtype).cuda()[:, None]
    T = v.shape[0]
    k = torch.ones_like(v)
    kc, vc, sc = moe.alloc_fp8_cache(T // 16, Hkv, 16, D)
    ws = moe.alloc_attn_workspace(T, 1, 1, 1, D)
    moe.rope_append_fp8(v.clone(), k, v, torch.zeros(4, 0, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda"),
                        ints([list(range(T // 16))]), ints([0, T]), ints([T]), kc, vc, sc, workspace=ws)
    assert moe.read_status(ws) == 0
    got = c8.values(vc)[:, 0].reshape(T, D)
    for b in range(T // 16):
        y = v[16 * b:16 * b + 16, 0].double().cpu()
        e = c8.scale_of(float(y.nan_to_num(0.0, float("inf"), -float("inf")).abs().max()))
        assert float(sc[b, 0, 0, 1]) == e
        w = c8.round8(y / e)
        assert torch.equal(got[16 * b:16 * b + 16].nan_to_num(1e9), w.nan_to_num(1e9)), b
    assert bool((sc[..., 0] == 2.0 ** -8).all())          # of ones


def test_token_by_token_stays_within_the_growth_of_scales():
    """A sequence grown by single tokens: a value is rounded once and once more, with half a step of the subnormal
    codes, each time its block's scale grows, which at most doubles the sum of those: 2^-4 of it and a step of 2^-9 of
    the block's scale."""
    g = gen_of(3)
    T, Hkv, D, page = 50, 2, 128, 16
    k = rand(g, T, Hkv, D) * torch.exp2(torch.arange(T, device="cuda") % 16 / 3.0)[:, None, None].to(BF)
    v = rand(g, T, Hkv, D) * torch.exp2(torch.arange(T, device="cuda") % 16 / 2.0)[:, None, None].to(BF)
    kc, vc, sc = moe.alloc_fp8_cache(5, Hkv, page, D)
    pages, none = ints([[4, 0, 2, 1]]), torch.zeros(4, 0, device="cuda")
    for t in range(T):
        moe.rope_append_fp8(k[t:t + 1], k[t:t + 1], v[t:t + 1], none, ints([0]), pages, ints([0, 1]), ints([t + 1]), kc,
                            vc, sc)
    for x, (c, y) in enumerate(((kc, k), (vc, v))):
        got = c8.rows(c, sc, x, pages[0], T)
        s = sc[pages[0].long()][..., x].double().repeat_interleave(16, 2).permute(1, 0, 2).reshape(Hkv, -1)[:, :T]
        want = y.double().transpose(0, 1)
        ref.check(got, want, 2.0 ** -4 * want.abs() + 2.0 ** -9 * s[..., None], "grown")
        for b in range(3):                                   # the scale that the whole block asks for
            for h in range(Hkv):
                top = float(want[h, 16 * b:16 * b + 16].abs().max())
                assert float(sc[pages[0, b], h, 0, x]) == c8.scale_of(top)


def test_what_is_out_of_range_is_reported_and_left():
    case = ([5, 20, 40], [30, 9, 3], 4, 2, 64, 32, False, False, 1, 16, BF)
    q, k, v, table, pos, pages, qs, lens, kc, vc, sc, (qn, kn), axes = append_case(case)
    ws = moe.alloc_attn_workspace(q.shape[0], 3, 4, 2, 64)

    def call(pages=pages, qs=qs, lens=lens, pos=pos):
        c = [x.clone() for x in (kc, vc, sc)]
        out = moe.rope_append_fp8(q, k, v, table, pos, pages, qs, lens, *c, workspace=ws)
        return c, out, moe.read_status(ws)

    def same(a, b, s):            # the rows of sequence s
        ids = pages[s, :(case[0][s] + case[1][s] + 15) // 16].long()
        return all(torch.equal(x.view(torch.uint8)[ids], y.view(torch.uint8)[ids]) for x, y in zip(a[:2], b[:2]))
    clean, out, status = call()
    assert status == 0
    for what in ("page", "negative page", "length", "too long", "short"):
        p, n = pages.clone(), lens.clone()
        if "page" in what:
            p[1, 1] = -1 if "neg" in what else kc.shape[0]
        else:
            n[1] = {"length": -1, "too long": 1 << 20, "short": 8}[what]
        got, o, status = call(p, lens=n)
        assert status == MOE_ERR_DEVICE, what
        assert same(got, clean, 0) and same(got, clean, 2) and torch.equal(o, out), what
        if "page" not in what:                               # nothing of the second was written
            assert same(got, [kc, vc, sc], 1)
    # rows that no sequence has: only their queries are written
    got, o, status = call(qs=ints([0, 30, 39, 39]), lens=ints([35, 29, 40]))
    assert status == MOE_ERR_DEVICE and same(got, clean, 0) and same(got, clean, 1) and same(got, [kc, vc, sc], 2)
    assert torch.equal(o, out)
    assert call(qs=ints([0, 30, 20, 42]))[2] == MOE_ERR_DEVICE
    bad = pos.clone()
    bad[35] = MAX_POS
    got, o, status = call(pos=bad)
    assert status == MOE_ERR_DEVICE and same(got, clean, 0) and same(got, clean, 2)


def test_a_token_without_a_position_leaves_its_row_and_the_scales():
    """Its key and its value stay as they were, as in the 16-bit append, and its size counts for no scale."""
    case = ([5, 20, 40], [30, 9, 3], 4, 2, 64, 32, False, False, 1, 16, BF)
    q, k, v, table, pos, pages, qs, lens, kc, vc, sc, (qn, kn), axes = append_case(case)
    k, v = k.contiguous(), v.contiguous()
    k[35], v[35] = 0, 0                                      # sequence 1: its token 25, on page 1, row 9
    clean = [x.clone() for x in (kc, vc, sc)]
    moe.rope_append_fp8(q, k, v, table, pos, pages, qs, lens, *clean)
    k[35], v[35] = 3000, -3000
    bad = pos.clone()
    bad[35] = -1
    ws = moe.alloc_attn_workspace(q.shape[0], 3, 4, 2, 64)
    got = [x.clone() for x in (kc, vc, sc)]
    moe.rope_append_fp8(q, k, v, table, bad, pages, qs, lens, *got, workspace=ws)
    assert moe.read_status(ws) == MOE_ERR_DEVICE
    assert torch.equal(got[2], clean[2])
    for x, y, before in zip(got, clean, (kc, vc)):
        x, y, before = (t.view(torch.uint8).clone() for t in (x, y, before))
        p = int(pages[1, 1])
        assert torch.equal(x[p, :, 9], before[p, :, 9])
        x[p, :, 9] = y[p, :, 9]
        assert torch.equal(x, y)


def test_captured_and_on_another_stream():
    case = APPEND[2]
    q, k, v, table, pos, pages, qs, lens, kc, vc, sc, (qn, kn), axes = append_case(case)
    first = [x.clone() for x in (kc, vc, sc)]
    ws = moe.alloc_attn_workspace(q.shape[0], 2, case[2], case[3], case[4])
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")

    def call(cache, stream=None):
        return moe.rope_append_fp8(q, k, v, table, pos, pages, qs, lens, *cache, qn, kn, axes=axes, q_out=out, workspace=ws,
                                   stream=stream)
    call([kc, vc, sc])
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    again = [x.clone() for x in first]
    with torch.cuda.graph(graph):
        call(again)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = [x.clone() for x in first]
    side.wait_stream(torch.cuda.current_stream())
    call(there, side)
    side.synchronize()
    for cache in (again, there):
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache[:2], (kc, vc)))
        assert torch.equal(cache[2], sc)


def test_no_tokens():
    kc, vc, sc = moe.alloc_fp8_cache(2, 1, 16, 64)
    q = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    k = torch.empty(0, 1, 64, dtype=BF, device="cuda")
    table = moe.rope_table(10, 64)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out = moe.rope_append_fp8(q, k, k, table, none, ints([[0, 1]]), ints([0, 0]), ints([3]), kc, vc, sc)
    assert out.shape == (0, 2, 64)
