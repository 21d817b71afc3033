"""GPU tests of attention over a cache in 8 bits whose values differ in scale from
one end of the range to the other, with bounds for each output by itself: what a
row's keys of some weight and size contribute is right whatever other keys,
blocks of scales and later tokens hold."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_reference as ref  # noqa: E402
import cache8_reference as c8  # noqa: E402
from test_gpu_attention import BF, HF, gen_of, ints, rand, starts  # noqa: E402
from test_gpu_attention_fp8 import pool, rows  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


def attend(q, k, v, scale, seen, prefill, shared=0):
    """Outputs and log-sums in 64 bits, and bounds relative to sum p |v|, element by element.

    A logit's error as in attn_reference, with three more fp32 roundings of exponents below 2^6 (3 * 2^-19 ln 2) and, in
    prefill, the query parts' (cache8_reference).  P rounds once, in prefill to the element type, in decode to f16; f16
    below 2^-14 is on a grid of 2^-24, and the P of a row's largest weight so far is at least 1 (in decode, with the scale
    of the values at hand), so a weight e (1 for the largest) is off by min(e, 2^-25).  In decode bf16 queries come to
    f16, elements below 2^-28 of the largest off by 2^-39 of it.
    Values are exact in bf16 and in decode; in f16 prefill on a grid of 2^-24, as the outputs are.
    shared: the first keys are a prefix's, which decode reads as prefill does."""
    n, Hq, D = q.shape
    group, m, half = Hq // k.shape[0], k.shape[1], q.dtype == HF
    out, lse = torch.zeros(n, Hq, D, dtype=torch.float64, device=q.device), torch.zeros(n, Hq, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for h in range(Hq):
        x, kk, vv = q[:, h].double(), k[h // group], v[h // group]
        s, mag = x @ kk.T * scale, x.abs() @ kk.abs().T * abs(scale)
        off = (D + 4) * 2.0 ** -24 * mag + 3 * 2.0 ** -19 * math.log(2)
        big = x.abs().amax(1, keepdim=True)
        if prefill or shared:
            fine = (x.abs() < 2.0 ** (-6.8 if half else -9.8) * big).double()
            off = off + 2.0 ** -17.8 * big * abs(scale) * (fine @ kk.abs().T)
        if not prefill:
            off = off + 2.0 ** -39 * big * abs(scale) * kk.abs().sum(1)
        if seen is not None:
            s, off = s.masked_fill(~seen, -math.inf), off.masked_fill(~seen, 0.0)
        e = torch.exp(s - s.amax(1, keepdim=True))
        total = e.sum(1, keepdim=True)
        lost = e.clamp(max=2.0 ** -25)
        if not half:                                        # bf16 P has fp32's range
            lost[:, :m if prefill else shared] = 0.0
        p, summed = e / total, (m + 16) * 2.0 ** -24
        out[:, h] = p @ vv
        lse[:, h] = (s.amax(1, keepdim=True) + total.log())[:, 0]
        delta = off.amax(1, keepdim=True)
        rounds = ref.U[q.dtype] if prefill or shared else ref.U[HF]
        tol_o[:, h] = (ref.U[q.dtype] * out[:, h].abs() + (rounds + 4 * delta + 2 * summed) * (p @ vv.abs())
                       + lost / total @ vv.abs() + (2.0 ** -24 if half else 0.0) + 1e-35)
        tol_l[:, h] = 2 * delta[:, 0] + summed + 2.0 ** -21 * (4 + lse[:, h].abs())
    return out, lse, tol_o, tol_l


def check(kernel, q, kc, vc, sc, table, q_lens, kv_lens):
    """Prefill of the rows, or decode of every sequence's last row."""
    Hq, D = q.shape[1:]
    scale = D ** -0.5
    ws = moe.alloc_attn_workspace(q.shape[0], len(q_lens), Hq, kc.shape[1], D)
    if kernel == "decode":
        q = q[torch.tensor(q_lens, device="cuda").cumsum(0) - 1].contiguous()
        q_lens = [1] * len(q_lens)
    lse = torch.empty(q.shape[0], Hq, device="cuda")
    if kernel == "decode":
        out = moe.attn_decode_fp8(q, kc, vc, sc, table, ints(kv_lens), scale=scale, lse=lse, workspace=ws)
    else:
        out = moe.attn_prefill_paged_fp8(q, kc, vc, sc, table, starts(q_lens), ints(kv_lens), scale=scale, lse=lse,
                                         workspace=ws)
    assert moe.read_status(ws) == 0
    at = 0
    for s, (n, m) in enumerate(zip(q_lens, kv_lens)):
        k, v = rows(kc, vc, sc, table[s], m)
        o, le, to, tl = attend(q[at:at + n], k, v, scale, ref.causal(n, m, q.device), kernel == "prefill")
        ref.check(out[at:at + n], o, to, f"sequence {s}")
        ref.check(lse[at:at + n], le, tl, f"log-sums of sequence {s}")
        at += n


def setup(kv_lens, q_lens, Hq, Hkv, D, page, dtype, seed):
    """Keys whose logits are small but for what element 0 adds (queries have 8 there, keys 0)."""
    kc, vc, sc, table, _ = pool(kv_lens, page, Hkv, D, seed)
    q = rand(gen_of(seed + 1), sum(q_lens), Hq, D, dtype=dtype)
    q[..., 0] = 8
    kc.view(torch.uint8)[..., 0] = 0
    sc[..., 0] = torch.where(sc[..., 0].isnan(), sc[..., 0], torch.full_like(sc[..., 0], 2.0 ** -7))
    return q, kc, vc, sc, table


def put(cache, table, s, j, head, row):
    """A key's or value's codes (or one of them)."""
    page = cache.shape[2]
    where, what = row
    cache[int(table[s, j // page]), head, j % page, where] = torch.as_tensor(what, device="cuda", dtype=torch.float32).to(c8.F8)


def set_scale(sc, table, s, block, head, which, exponent):
    per = sc.shape[2]
    sc[int(table[s, block // per]), head, block % per, which] = 2.0 ** exponent


SHAPES = [(64, BF), (64, HF), (128, BF), (128, HF)]
KERNELS = ["decode", "prefill"]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("D,dtype", SHAPES)
@pytest.mark.parametrize("low", [-8, -18, -24])
def test_a_large_value_without_weight(kernel, D, dtype, low):
    """The first key's value is as large as can be and its weight 2^-57; the keys beside it have values of 0; all later
    ones have a scale that is 2^15 to 2^31 smaller, and are the output."""
    kv_lens, q_lens, Hq, Hkv, page = [600, 40], [70, 3], 8, 2, 32
    q, kc, vc, sc, table = setup(kv_lens, q_lens, Hq, Hkv, D, page, dtype, 101)
    for s, m in enumerate(kv_lens):
        for h in range(Hkv):
            for b in range((m + 15) // 16):
                set_scale(sc, table, s, b, h, 1, low)
            set_scale(sc, table, s, 0, h, 1, 7)
            for j in range(1, 16):
                put(vc, table, s, j, h, (slice(None), 0.0))
            # -39 in the logit: 8 * code * 2^e * D^-1/2, the block's other keys 0 there
            set_scale(sc, table, s, 0, h, 0, -3)
            for j in range(1, 16):
                put(kc, table, s, j, h, (slice(None), 0.0))
            put(kc, table, s, 0, h, (0, -448.0 if D == 128 else -320.0))
    check(kernel, q, kc, vc, sc, table, q_lens, kv_lens)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("D,dtype", SHAPES)
def test_blocks_of_zeros_under_a_large_scale(kernel, D, dtype):
    """Every other block of 16 has the largest scale and values of 0 (but for one without weight), the others the
    smallest: half of the weight lies on each."""
    kv_lens, q_lens, Hq, Hkv, page = [300, 130], [40, 130], 4, 1, 64
    q, kc, vc, sc, table = setup(kv_lens, q_lens, Hq, Hkv, D, page, dtype, 111)
    for s, m in enumerate(kv_lens):
        for b in range((m + 15) // 16):
            set_scale(sc, table, s, b, 0, 1, 7 if b % 2 == 0 else -24)
            if b % 2 == 0:
                for j in range(16 * b, min(16 * b + 16, m)):
                    put(vc, table, s, j, 0, (slice(None), 0.0))
    check(kernel, q, kc, vc, sc, table, q_lens, kv_lens)


@pytest.mark.parametrize("D,dtype", SHAPES)
@pytest.mark.parametrize("order", ["small first", "large first"])
def test_a_row_does_not_depend_on_later_tokens(D, dtype, order):
    """Causal rows of one block of keys: the first 64 tokens' values have the smallest scale, those behind them the
    largest (and the other way round)."""
    n, Hq, Hkv, page = 128, 8, 2, 16
    q, kc, vc, sc, table = setup([n], [n], Hq, Hkv, D, page, dtype, 121)
    for h in range(Hkv):
        for b in range(n // 16):
            set_scale(sc, table, 0, b, h, 1, (-24 if b < 4 else 7) if order == "small first" else (7 if b < 4 else -24))
    check("prefill", q, kc, vc, sc, table, [n], [n])
    # and the first rows are the same as of a call without the others
    some = moe.attn_prefill_paged_fp8(q, kc, vc, sc, table, ints([0, n]), ints([n]))[:64]
    alone = moe.attn_prefill_paged_fp8(q[:64].contiguous(), kc, vc, sc, table, ints([0, 64]), ints([64]))
    assert torch.equal(some, alone)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("D,dtype", SHAPES)
@pytest.mark.parametrize("spread", [4, 14])
def test_scales_of_any_size(kernel, D, dtype, spread):
    kv_lens, q_lens, Hq, Hkv, page = [1000, 50, 200], [60, 50, 1], 24, 3, 16
    kc, vc, sc, table, _ = pool(kv_lens, page, Hkv, D, 131, spread=spread)
    q = rand(gen_of(132), sum(q_lens), Hq, D, dtype=dtype, mul=4.0)
    check(kernel, q, kc, vc, sc, table, q_lens, kv_lens)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("D,dtype", SHAPES)
@pytest.mark.parametrize("gap", [0, 60])
def test_a_heavy_key_without_a_value(kernel, D, dtype, gap):
    """A key of 2^12 times the others' weight whose value is 0, first or in the middle, under the largest scale; the
    others under the smallest."""
    kv_lens, q_lens, Hq, Hkv, page = [500], [20], 8, 2, 64
    q, kc, vc, sc, table = setup(kv_lens, q_lens, Hq, Hkv, D, page, dtype, 141)
    for h in range(Hkv):
        for b in range(32):
            set_scale(sc, table, 0, b, h, 1, -24)
        block = gap // 16
        set_scale(sc, table, 0, block, h, 1, 7)
        set_scale(sc, table, 0, block, h, 0, -5)
        for j in range(16 * block, 16 * block + 16):
            put(vc, table, 0, j, h, (slice(None), 0.0))
            put(kc, table, 0, j, h, (slice(None), 0.0))
        put(kc, table, 0, gap, h, (0, 8.3 * D ** 0.5 / 8 * 2.0 ** 5))          # 8.3 in the logit
    check(kernel, q, kc, vc, sc, table, q_lens, kv_lens)


@pytest.mark.parametrize("D,dtype", SHAPES)
def test_an_infinite_query_over_keys_that_it_hides(D, dtype):
    """Decode: logits that are all -inf, beside the largest finite elements of the query against keys of the other sign,
    give 0 and a log-sum of -inf; the other heads are as without."""
    kv_lens, Hq, Hkv, page = [300, 40], 8, 2, 16
    kc, vc, sc, table, _ = pool(kv_lens, page, Hkv, D, 161)
    for s, m in enumerate(kv_lens):
        for j in range(m):
            for h in range(Hkv):
                put(kc, table, s, j, h, (0, -2.0))
                put(kc, table, s, j, h, (1, 3.0))
    q = rand(gen_of(162), 2, Hq, D, dtype=dtype)

    def call():
        lse = torch.empty(2, Hq, device="cuda")
        return moe.attn_decode_fp8(q, kc, vc, sc, table, ints(kv_lens), lse=lse), lse
    want, lse = call()
    q[1, 3] = 1
    q[1, 3, 0], q[1, 3, 1] = math.inf, torch.finfo(dtype).max
    got, lse1 = call()
    assert bool((got[1, 3] == 0).all()) and float(lse1[1, 3]) == -math.inf
    got[1, 3], lse1[1, 3] = want[1, 3], lse[1, 3]
    assert torch.equal(got, want) and torch.equal(lse1, lse)


@pytest.mark.parametrize("D,dtype", SHAPES)
def test_behind_a_prefix(D, dtype):
    """Decode behind a shared prefix: rows of queries with an element 2^12 times the others, and one with an infinity,
    whose head is NaN there and nowhere else."""
    kv_lens, shared, Hq, Hkv, page = [300, 20, 0], 500, 8, 2, 16
    kc, vc, sc, table, pre = pool(kv_lens, page, Hkv, D, 151, prefix=shared, spread=10)
    q = rand(gen_of(152), 3, Hq, D, dtype=dtype)
    high = torch.arange(Hq, device="cuda")
    q[:, high, high * 5] = 2.0 ** 12
    scale = 0.02 * D ** -0.5
    ws = moe.alloc_attn_workspace(3, 3, Hq, Hkv, D)

    def call():
        lse = torch.empty(3, Hq, device="cuda")
        out = moe.attn_decode_fp8(q, kc, vc, sc, table, ints(kv_lens), pre, shared, scale=scale, lse=lse, workspace=ws)
        assert moe.read_status(ws) == 0
        return out, lse
    out, lse = call()
    for b, n in enumerate(kv_lens):
        k, v = rows(kc, vc, sc, table[b], n)
        pk, pv = rows(kc, vc, sc, pre, shared)
        k, v = torch.cat([pk, k], 1), torch.cat([pv, v], 1)
        o, le, to, tl = attend(q[b:b + 1], k, v, scale, None, False, shared)
        ref.check(out[b:b + 1], o, to, f"out of row {b}")
        ref.check(lse[b:b + 1], le, tl, f"lse of row {b}")
    q[1, 3, 7] = math.inf
    got = call()[0]
    assert bool(got[1, 3].isnan().all())
    got[1, 3] = out[1, 3]
    assert torch.equal(got, out)
