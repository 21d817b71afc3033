"""CPU tests of the largest sizes of the operators around the paged cache: a size
whose indices, rounded up to a tile, would pass 32 bits is refused (none of these
calls reaches a GPU)."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_attention_host import C, FAKE, H, UNSUPPORTED, WORKSPACE  # noqa: E402
from test_cache_host import C8  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402
from expert_layer_gb300 import _build  # noqa: E402

MOST = (1 << 31) - (1 << 16)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.lib()


def test_key_weights(lib):
    def call(room=100, n=2, Hkv=2):
        return lib.moe_attn_key_weights(H(), FAKE, 8, 16, FAKE, 4, FAKE, FAKE, n, 4, 2 * Hkv, Hkv, 128, 0, 1, 0.1, FAKE, FAKE,
                                        room, FAKE, 16, None)
    assert call(room=MOST) == WORKSPACE
    assert call(room=MOST + 1) == UNSUPPORTED and call(room=(1 << 31) - 1) == UNSUPPORTED
    assert call(n=MOST // 2) == WORKSPACE and call(n=MOST // 2 + 1) == UNSUPPORTED
    assert call(n=1 << 20, Hkv=1 << 12) == UNSUPPORTED                    # a product past 32 bits


def test_evict(lib):
    def call(room=100, budget=64, out_pages=4, n=2, Hkv=2, page=16):
        return lib.moe_kv_evict(C(size=page), FAKE, 4, FAKE, FAKE, room, FAKE, out_pages, budget, 4, 8, n, Hkv, 128, FAKE, FAKE,
                                FAKE, FAKE, 16, None)
    assert call(room=MOST) == WORKSPACE and call(room=MOST + 1) == UNSUPPORTED
    wide = 1 << 23                                                        # pages of 256: 2^31 rows
    assert call(budget=MOST, out_pages=wide, page=256) == WORKSPACE
    assert call(budget=MOST + 1, out_pages=wide, page=256) == UNSUPPORTED
    assert call(n=MOST // 2) == WORKSPACE and call(n=MOST // 2 + 1) == UNSUPPORTED
    assert call(n=1 << 20, Hkv=1 << 12) == UNSUPPORTED


def test_attention_over_8_bits(lib):
    def prefill(wide, page):
        return lib.moe_attn_prefill_paged_fp8(H(), C8(size=page), FAKE, wide, FAKE, FAKE, 2, 4, 4, 2, 128, 0, 1, 0.1, FAKE, None,
                                              FAKE, 16, None)

    def decode(wide, page):
        return lib.moe_attn_decode_fp8(H(), C8(size=page), FAKE, wide, FAKE, None, 0, 4, 4, 2, 128, 0, 0.1, FAKE, None, FAKE, 16,
                                       None)
    for call in (prefill, decode):
        for page in (16, 256):
            assert call(MOST // page, page) == WORKSPACE
            assert call(MOST // page + 1, page) == UNSUPPORTED and call((1 << 31) - 1, page) == UNSUPPORTED
