"""GPU test of eviction whose new lengths replace the old ones."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_attention import ints  # noqa: E402
from test_gpu_key_weights import EVICT, evict_case  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


@pytest.mark.parametrize("case", [EVICT[1], EVICT[7], EVICT[9], EVICT[10]], ids=lambda c: f"{len(c[0])}x{max(c[0])}-to{c[1]}")
def test_new_lengths_in_place_of_the_old(case):
    """Every head of a sequence selects by the old length, whichever is done first (1100 sequences are more heads than
    blocks of the grid)."""
    kv_lens, budget, first, last, Hkv, D, page, dtype, kind, more = case
    got = []
    for same in (False, True):
        kc, vc, table, out_table, w = evict_case(case)
        lens = ints(kv_lens)
        ws = moe.alloc_attn_workspace(0, len(kv_lens), Hkv, Hkv, D)
        out = moe.kv_evict(kc, vc, table, lens, w, out_table, budget, keep_first=first, keep_last=last,
                           new_lens=lens if same else None, workspace=ws)
        assert moe.read_status(ws) == 0
        assert (out[0] is lens) == same
        got.append([x.view(torch.int32) for x in out] + [x.view(torch.int16) for x in (kc, vc)])
    assert got[0][0].tolist() == [min(n, budget) for n in kv_lens]
    assert all(torch.equal(a, b) for a, b in zip(*got))
