"""CPU tests of the operators around the paged cache: refusals of bad arguments
(none of these calls reaches a GPU), the axes of rotated pairs, the 8-bit
reference against PyTorch's own type."""
import ctypes
import os
import struct
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import cache8_reference as c8  # noqa: E402
from test_attention_host import C, FAKE, H, INVALID, MIS, UNSUPPORTED, WORKSPACE  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402
from expert_layer_gb300 import _build  # noqa: E402

BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.lib()


def C8(k=1 << 20, v=1 << 20, scales=1 << 20, pages=8, size=16):
    return struct.pack("=QQQii", k, v, scales, pages, size)      # moe_kv_cache_fp8


def test_rope_append_axes_refusals(lib):
    def call(axes=FAKE, n_axes=3, rot=128, T=4, pos=FAKE):
        return lib.moe_rope_append_axes(H(), H(), H(), None, None, 1e-6, FAKE, 64, rot, 0, pos, axes, n_axes, FAKE, T, 4, 2,
                                        128, 0, FAKE, C(), FAKE, 16, None)
    assert call() == WORKSPACE and call(axes=None, n_axes=0) == WORKSPACE     # everything before it is fine
    assert call(T=0) == 0
    assert call(n_axes=0) == INVALID
    assert call(n_axes=5) == UNSUPPORTED
    assert call(axes=MIS) == UNSUPPORTED
    assert call(pos=None) == INVALID


def test_rope_append_fp8_refusals(lib):
    def call(q=None, k=None, table=FAKE, rot=128, pos=FAKE, axes=None, n_axes=0, pages=FAKE, wide=4, qs=FAKE, lens=FAKE, n=2,
             T=4, Hq=4, Hkv=2, D=128, dtype=0, out=FAKE, cache=None, ws=FAKE, room=16):
        return lib.moe_rope_append_fp8(q or H(), k or H(), H(), None, None, 1e-6, table, 64, rot, 0, pos, axes, n_axes, pages,
                                       wide, qs, lens, n, T, Hq, Hkv, D, dtype, out, cache or C8(), ws, room, None)
    assert call() == WORKSPACE
    assert call(T=0) == 0
    assert call(n=0) == INVALID and call(n=-1) == INVALID and call(n=1 << 29) == UNSUPPORTED
    assert call(wide=0) == INVALID
    assert call(D=96) == UNSUPPORTED and call(Hq=5) == INVALID and call(dtype=2) == INVALID
    assert call(rot=24) == UNSUPPORTED and call(rot=144) == INVALID
    assert call(axes=FAKE, n_axes=5) == UNSUPPORTED and call(axes=FAKE, n_axes=0) == INVALID
    for name in ("pages", "qs", "lens", "pos"):
        assert call(**{name: None}) == INVALID and call(**{name: MIS}) == UNSUPPORTED, name
    assert call(out=None) == INVALID and call(ws=None) == INVALID and call(table=None) == INVALID
    assert call(cache=C8(k=0)) == INVALID and call(cache=C8(scales=0)) == INVALID
    assert call(cache=C8(v=(1 << 20) + 8)) == UNSUPPORTED and call(cache=C8(scales=(1 << 20) + 4)) == UNSUPPORTED
    assert call(cache=C8(size=24)) == UNSUPPORTED and call(cache=C8(size=512)) == UNSUPPORTED
    assert call(cache=C8(pages=0)) == INVALID
    assert call(k=H(tok=511)) == UNSUPPORTED


def test_attention_fp8_refusals(lib):
    def prefill(cache=None, wide=4, scale=0.1, ws=FAKE, out=FAKE, T=4, n=2, qs=FAKE):
        return lib.moe_attn_prefill_paged_fp8(H(), cache or C8(), FAKE, wide, qs, FAKE, n, T, 4, 2, 128, 0, 1, scale, out, None,
                                              ws, 16, None)

    def decode(cache=None, wide=4, scale=0.1, ws=FAKE, out=FAKE, T=4, prefix=None, prefix_len=0):
        return lib.moe_attn_decode_fp8(H(), cache or C8(), FAKE, wide, FAKE, prefix, prefix_len, T, 4, 2, 128, 0, scale, out,
                                       None, ws, 16, None)
    for call in (prefill, decode):
        assert call() == WORKSPACE and call(T=0) == 0
        assert call(wide=0) == INVALID and call(scale=float("nan")) == INVALID
        assert call(out=None) == INVALID and call(ws=MIS) == UNSUPPORTED
        assert call(cache=C8(scales=0)) == INVALID and call(cache=C8(size=8)) == UNSUPPORTED
        assert call(cache=C8(scales=(1 << 20) + 8)) == UNSUPPORTED
    assert prefill(n=0) == INVALID and prefill(qs=None) == INVALID
    assert decode(prefix_len=-1) == INVALID and decode(prefix_len=5) == INVALID


def test_key_weights_refusals(lib):
    def call(k=FAKE, size=16, wide=4, n=2, T=4, D=128, dtype=0, scale=0.1, lse=FAKE, w=FAKE, room=100, qs=FAKE, ws=FAKE):
        return lib.moe_attn_key_weights(H(), k, 8, size, FAKE, wide, qs, FAKE, n, T, 4, 2, D, dtype, 1, scale, lse, w, room,
                                        ws, 16, None)
    assert call() == WORKSPACE and call(T=0) == 0
    assert call(k=None) == INVALID and call(k=MIS) == UNSUPPORTED and call(size=24) == UNSUPPORTED
    assert call(wide=0) == INVALID and call(n=0) == INVALID and call(room=0) == INVALID
    assert call(D=96) == UNSUPPORTED and call(dtype=3) == INVALID
    assert call(scale=float("inf")) == INVALID and call(scale=float("nan")) == INVALID
    for name in ("lse", "w", "qs", "ws"):
        assert call(**{name: None}) == INVALID and call(**{name: MIS}) == UNSUPPORTED, name


def test_evict_refusals(lib):
    def call(cache=None, wide=4, room=100, out_pages=4, budget=64, first=4, last=8, n=2, Hkv=2, D=128, lens=FAKE, w=FAKE,
             to=FAKE, kept=FAKE, ws=FAKE):
        return lib.moe_kv_evict(cache or C(), FAKE, wide, lens, w, room, to, out_pages, budget, first, last, n, Hkv, D, FAKE,
                                FAKE, kept, ws, 16, None)
    assert call() == WORKSPACE and call(n=0) == 0
    assert call(budget=0) == INVALID and call(budget=65) == INVALID            # more than the pages hold
    assert call(first=-1) == INVALID and call(last=-1) == INVALID and call(first=60, last=5) == INVALID
    assert call(first=BIG, last=BIG) == INVALID
    assert call(wide=0) == INVALID and call(room=0) == INVALID and call(out_pages=0) == INVALID
    assert call(D=32) == UNSUPPORTED and call(Hkv=0) == INVALID and call(n=-1) == INVALID
    assert call(cache=C(size=10)) == UNSUPPORTED
    for name in ("lens", "w", "to", "kept", "ws"):
        assert call(**{name: None}) == INVALID and call(**{name: MIS}) == UNSUPPORTED, name


def test_python_functions_refuse_what_is_not_theirs(lib):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for f in (moe.rope_append_fp8, moe.attn_prefill_paged_fp8, moe.attn_decode_fp8, moe.attn_key_weights):
        with pytest.raises(moe.MoEError):
            f(q, *[q] * 10)
        with pytest.raises(TypeError):
            f(q)
    with pytest.raises(moe.MoEError, match="k_cache must be a CUDA tensor"):
        moe.kv_evict(q, q, q, q, q, q, 8)
    with pytest.raises(moe.MoEError, match="bfloat16 or float16"):
        moe.kv_evict(q.float(), q, q, q, q, q, 8)
    for bad in (dict(pages=0, Hkv=1, page_size=16, D=64), dict(pages=1, Hkv=1, page_size=24, D=64)):
        with pytest.raises(moe.MoEError):
            moe.alloc_fp8_cache(**bad, device="cpu")
    k, v, s = moe.alloc_fp8_cache(3, 2, 32, 64, device="cpu")
    assert k.dtype == v.dtype == torch.float8_e4m3fn and k.shape == v.shape == (3, 2, 32, 64)
    assert s.dtype == torch.float32 and s.shape == (3, 2, 2, 2)


def test_rope_axes():
    assert moe.rope_axes(16, (3, 2, 3), device="cpu").tolist() == [0, 0, 0, 1, 1, 2, 2, 2]
    assert moe.rope_axes(16, (4, 2, 2), True, device="cpu").tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    assert moe.rope_axes(8, (0, 4), device="cpu").tolist() == [1] * 4
    assert moe.rope_axes(0, (0,), device="cpu").tolist() == []
    for bad in ((16, (3, 2)), (16, (9, -1)), (10, (1, 1, 1, 1, 1)), (16, ())):
        with pytest.raises(moe.MoEError):
            moe.rope_axes(*bad, device="cpu")


def test_the_8_bit_reference_rounds_as_the_type_does():
    x = torch.cat([torch.randn(20000, dtype=torch.float64) * s for s in (0.01, 1.0, 100.0)])
    every = torch.arange(256, dtype=torch.uint8).view(c8.F8).double()
    every = every[~every.isnan()]
    between = (every.sort().values[:-1] + every.sort().values[1:]) / 2          # ties
    x = torch.cat([x.clamp(-448, 448), every, between])
    assert torch.equal(c8.round8(x), x.float().to(c8.F8).double())
    assert float(c8.round8(torch.tensor(1e9))) == 448 and bool(c8.round8(torch.tensor(float("nan"))).isnan())
    assert c8.scale_of(448.0) == 1 and c8.scale_of(448.0000001) == 2 and c8.scale_of(0.0) == 2.0 ** -24
    assert c8.scale_of(1e9) == 128
