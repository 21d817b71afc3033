"""CPU tests of the attention entry points: refusals of bad arguments (none
of these calls reaches a GPU), workspace sizes, and the rotary table."""
import ctypes
import math
import struct

import pytest
import torch

import expert_layer_gb300 as moe
from expert_layer_gb300 import _build

P = ctypes.c_void_p
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.lib()


def H(ptr=1 << 20, tok=512, head=128):
    return struct.pack("=Qqq", ptr, tok, head)          # moe_heads


def C(k=1 << 20, v=1 << 20, pages=8, size=16):
    return struct.pack("=QQii", k, v, pages, size)      # moe_kv_cache


FAKE, MIS = P(1 << 20), P((1 << 20) + 2)      # never dereferenced: every case fails on the host


def rope(lib, q=None, k=None, v=None, qn=None, kn=None, eps=1e-6, table=FAKE, max_pos=64, rot=128, pos=FAKE, slots=FAKE,
         T=4, Hq=4, Hkv=2, D=128, dtype=0, out=FAKE, cache=None, ws=FAKE, n=None):
    n = 1 << 30 if n is None else n
    return lib.moe_rope_append(q or H(), k or H(), v or H(), qn, kn, eps, table, max_pos, rot, 0, pos, slots, T, Hq,
                               Hkv, D, dtype, out, cache or C(), ws, n, None)


def test_rope_append_refusals(lib):
    assert rope(lib, T=0) == 0                                    # an empty batch is fine
    assert rope(lib, T=-1) == INVALID
    assert rope(lib, Hq=5) == INVALID                             # Hq not a multiple of Hkv
    assert rope(lib, D=96) == UNSUPPORTED
    assert rope(lib, Hq=258, Hkv=2) == UNSUPPORTED                # more than 128 heads on one
    assert rope(lib, dtype=2) == INVALID
    assert rope(lib, rot=136) == INVALID
    assert rope(lib, rot=24) == UNSUPPORTED
    assert rope(lib, max_pos=0) == INVALID
    assert rope(lib, eps=-1.0) == INVALID
    assert rope(lib, eps=float("nan")) == INVALID
    assert rope(lib, q=H(ptr=0)) == INVALID
    assert rope(lib, q=H(ptr=(1 << 20) + 8)) == UNSUPPORTED
    assert rope(lib, k=H(tok=511)) == UNSUPPORTED
    assert rope(lib, k=H(head=0)) == INVALID
    assert rope(lib, table=None) == INVALID
    assert rope(lib, pos=None) == INVALID
    assert rope(lib, slots=MIS) == UNSUPPORTED
    assert rope(lib, out=MIS) == UNSUPPORTED
    assert rope(lib, qn=P((1 << 20) + 4)) == UNSUPPORTED
    assert rope(lib, cache=C(k=0)) == INVALID
    assert rope(lib, cache=C(size=24)) == UNSUPPORTED
    assert rope(lib, cache=C(size=8)) == UNSUPPORTED
    assert rope(lib, cache=C(pages=0)) == INVALID
    assert rope(lib, cache=C(pages=1 << 27)) == UNSUPPORTED       # 2^31 rows
    assert rope(lib, ws=None) == INVALID
    assert rope(lib, n=moe.attn_workspace_size(4, 0, 4, 2, 128) - 1) == WORKSPACE


def prefill(lib, q=None, k=None, v=None, qs=FAKE, ks=FAKE, n_seq=2, T=8, Tk=8, Hq=4, Hkv=2, D=128, dtype=0, scale=0.1,
            out=FAKE, lse=None, ws=FAKE, n=1 << 40):
    return lib.moe_attn_prefill(q or H(), k or H(), v or H(), qs, ks, n_seq, T, Tk, Hq, Hkv, D, dtype, 1, scale, out,
                                lse, ws, n, None)


def test_prefill_refusals(lib):
    assert prefill(lib, T=0) == 0
    assert prefill(lib, Tk=-1) == INVALID
    assert prefill(lib, n_seq=0) == INVALID
    assert prefill(lib, n_seq=-1) == INVALID
    assert prefill(lib, D=256) == UNSUPPORTED
    assert prefill(lib, T=1 << 30) == UNSUPPORTED                 # T * Hq past 2^31
    assert prefill(lib, dtype=7) == INVALID
    assert prefill(lib, qs=None) == INVALID
    assert prefill(lib, ks=None) == INVALID
    assert prefill(lib, k=H(ptr=0)) == INVALID
    assert prefill(lib, v=H(tok=4)) == UNSUPPORTED
    assert prefill(lib, out=None) == INVALID
    assert prefill(lib, lse=MIS) == UNSUPPORTED
    assert prefill(lib, scale=float("nan")) == INVALID
    assert prefill(lib, scale=float("inf")) == INVALID
    assert prefill(lib, n=moe.attn_workspace_size(8, 2, 4, 2, 128) - 1) == WORKSPACE


def paged(lib, q=None, cache=None, table=FAKE, wide=4, qs=FAKE, lens=FAKE, n_seq=2, T=8, Hq=4, Hkv=2, D=128, ws=FAKE,
          n=1 << 40):
    return lib.moe_attn_prefill_paged(q or H(), cache or C(), table, wide, qs, lens, n_seq, T, Hq, Hkv, D, 0, 1, 0.1,
                                      FAKE, None, ws, n, None)


def test_prefill_paged_refusals(lib):
    assert paged(lib, T=0) == 0
    assert paged(lib, wide=0) == INVALID
    assert paged(lib, table=None) == INVALID
    assert paged(lib, lens=None) == INVALID
    assert paged(lib, qs=MIS) == UNSUPPORTED
    assert paged(lib, cache=C(size=512)) == UNSUPPORTED
    assert paged(lib, cache=C(v=(1 << 20) + 8)) == UNSUPPORTED
    assert paged(lib, ws=P((1 << 20) + 8)) == UNSUPPORTED
    assert paged(lib, n=16) == WORKSPACE


def decode(lib, cache=None, table=FAKE, wide=4, lens=FAKE, pre=None, pre_len=0, B=2, Hq=4, Hkv=2, D=128, n=1 << 40):
    return lib.moe_attn_decode(H(), cache or C(), table, wide, lens, pre, pre_len, B, Hq, Hkv, D, 0, 0.1, FAKE, None,
                               FAKE, n, None)


def test_decode_refusals(lib):
    assert decode(lib, B=0) == 0
    assert decode(lib, B=-3) == INVALID
    assert decode(lib, wide=0) == INVALID
    assert decode(lib, pre_len=-1) == INVALID
    assert decode(lib, pre_len=10) == INVALID                     # a prefix without its pages
    assert decode(lib, lens=None) == INVALID
    assert decode(lib, Hq=6, Hkv=4) == INVALID
    assert decode(lib, D=32) == UNSUPPORTED
    assert decode(lib, wide=1 << 30, cache=C(pages=1 << 20)) == UNSUPPORTED   # 2^31 slices of 16 keys
    assert decode(lib, n=0) == WORKSPACE


def test_workspace_size(lib):
    assert moe.attn_workspace_size(1, 1, 32, 4, 128) > 0
    assert moe.attn_workspace_size(8192, 4, 32, 4, 128) >= moe.attn_workspace_size(1, 1, 32, 4, 128)
    assert moe.attn_workspace_size(1, 1, 32, 5, 128) == 0
    assert moe.attn_workspace_size(1, 1, 32, 4, 80) == 0
    assert moe.attn_workspace_size(-1, 1, 32, 4, 128) == 0
    with pytest.raises(moe.MoEError):
        moe.alloc_attn_workspace(1, 1, 32, 5, 128)


def test_binding_rejects_before_the_library(lib):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    c = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(moe.MoEError, match="CUDA"):
        moe.attn_prefill(q, q[:, :2], q[:, :2], i, i)
    with pytest.raises(moe.MoEError, match="CUDA"):
        moe.attn_decode(q, c, c, i[None], i)
    with pytest.raises(moe.MoEError, match="bfloat16 or float16"):
        moe.attn_decode(q.float(), c, c, i[None], i)
    with pytest.raises(moe.MoEError, match="Tensor"):
        moe.rope_append(None, q, q, q, i, i, c, c)
    with pytest.raises(TypeError, match="kv_lens"):
        moe.attn_decode(q, c, c, i[None])
    with pytest.raises(TypeError, match="unexpected"):
        moe.attn_decode(q, c, c, i[None], i, softcap=3.0)
    with pytest.raises(TypeError, match="repeated"):
        moe.attn_prefill(q, q, q, i, i, q_starts=i)
    with pytest.raises(TypeError, match="at most"):
        moe.attn_prefill(*([q] * 12))


def test_rope_table_values():
    t = moe.rope_table(50, 32, base=500.0, device="cpu")
    assert t.shape == (50, 32) and t.dtype == torch.float32
    for p in (0, 1, 49):
        for i in (0, 3, 15):
            a = p * 500.0 ** (-2 * i / 32)
            assert abs(float(t[p, i]) - math.cos(a)) < 2.0 ** -23 and abs(float(t[p, 16 + i]) - math.sin(a)) < 2.0 ** -23
    # linear scaling by 4: position 4p has the angles of position p
    lin = moe.rope_table(50, 32, base=500.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin[40], t[10], atol=2.0 ** -22)
    # by parts: the fastest frequencies stay, the slowest are divided, both times 0.1 ln 8 + 1
    big = moe.rope_table(9000, 64, base=10000.0, device="cpu")
    yar = moe.rope_table(9000, 64, base=10000.0, scaling="by_parts", factor=8.0, original_max_pos=1024, device="cpu")
    mul = 0.1 * math.log(8.0) + 1
    assert torch.allclose(yar[:, 0], big[:, 0] * mul, atol=2.0 ** -21)
    assert torch.allclose(yar[8000, 31], big[1000, 31] * mul, atol=2.0 ** -21)
    assert torch.allclose(yar[8000, 63], big[1000, 63] * mul, atol=2.0 ** -21)
    for bad in (dict(rot=7), dict(max_pos=0), dict(base=1.0), dict(factor=0.5), dict(scaling="other"),
                dict(scaling="by_parts")):
        with pytest.raises(moe.MoEError):
            moe.rope_table(**{**dict(max_pos=8, rot=8, device="cpu"), **bad})
