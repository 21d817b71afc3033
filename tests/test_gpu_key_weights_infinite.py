"""GPU tests of the attention weight of keys that hold an infinity, in both of its
kernels (few rows of a sequence and head, and many) and for groups that do and do
not divide a tile of 128 rows."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_reference as ref  # noqa: E402
from test_gpu_attention import BF, HF, gen_of, ints, page_pool, rand, starts  # noqa: E402
from test_gpu_key_weights import weights_reference  # noqa: E402

import expert_layer_gb300 as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_layer_gb300 import _build
    _build.build()
    moe.lib()


def queries(T, Hq, D, dtype):
    """Element 0 above 1, so that an infinite element 0 of a key makes every row's logit infinite."""
    q = rand(gen_of(6), T, Hq, D, dtype=dtype, mul=2.5)
    q[..., 0] = q[..., 0].abs() + 1
    return q


# rows of each sequence: one goes to the warps' kernel, 150 (two row tiles and a part of one where G = 3 or more) to the
# tensor cores
@pytest.mark.parametrize("rows", [1, 150])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,D,dtype", [(1, 64, BF), (3, 64, HF), (6, 128, BF), (7, 64, BF), (8, 128, HF), (24, 128, BF)])
def test_keys_with_an_infinity(rows, causal, G, D, dtype):
    """A key whose logits are all -inf has a weight of 0 and its entry stays as it was; one of +inf under a finite
    log-sum gets an infinity, one that is NaN gets NaN; every other key's weight is what it is without them."""
    Hkv, page, kv_lens = 2, 32, [700, 400]
    q_lens = [rows, rows]
    kc, vc, table, _ = page_pool(kv_lens, page, Hkv, D, dtype, 5)
    q = queries(sum(q_lens), G * Hkv, D, dtype)
    gone, high, lost = [0, 33, 127, 128, 201], 140, 141               # of sequence 0; every row sees them
    pages = [int(x) for x in table[0, :22]]
    for j in gone:
        kc[pages[j // page], :, j % page, 0] = -math.inf
    lse = torch.empty(q.shape[0], G * Hkv, device="cuda")
    moe.attn_prefill_paged(q, kc, torch.zeros_like(kc), table, starts(q_lens), ints(kv_lens), causal=causal, lse=lse)
    assert bool(lse.isfinite().all())
    kc[pages[high // page], :, high % page, 0] = math.inf
    kc[pages[lost // page], :, lost % page, 3] = math.nan
    w = torch.rand(2, Hkv, 700, generator=gen_of(7), device="cuda")
    first = w.clone()
    ws = moe.alloc_attn_workspace(q.shape[0], 2, G * Hkv, Hkv, D)
    moe.attn_key_weights(q, kc, table, starts(q_lens), ints(kv_lens), lse, w, causal=causal, workspace=ws)
    assert moe.read_status(ws) == 0
    assert torch.equal(w[0][:, gone], first[0][:, gone])
    assert bool((w[0, :, high] == math.inf).all()) and bool(w[0, :, lost].isnan().all())
    clean = torch.where(kc.isfinite(), kc, torch.zeros_like(kc))
    want, tol = weights_reference(q, q_lens, kv_lens, clean, table, causal, D ** -0.5, lse, first)
    others = [j for j in range(700) if j not in gone + [high, lost]]
    ref.check(w[0][:, others], want[0][:, others], tol[0][:, others], "weights")
    ref.check(w[1], want[1], tol[1], "weights of the other sequence")


@pytest.mark.parametrize("rows", [1, 150])
def test_log_sums_without_a_weight(rows):
    """Log-sums of -inf (rows without keys) and of +inf give nothing; queries of rows without keys may be anything."""
    Hq, Hkv, D, page, q_lens, kv_lens = 12, 2, 64, 16, [rows, rows], [300, 200]
    kc, vc, table, _ = page_pool(kv_lens, page, Hkv, D, BF, 9)
    q = rand(gen_of(10), sum(q_lens), Hq, D)
    lse = rand(gen_of(11), sum(q_lens), Hq, dtype=torch.float32).abs() + 3
    lse[0], lse[-1, 2] = -math.inf, math.inf
    q[0, 3] = math.nan
    w = torch.zeros(2, Hkv, 300, device="cuda")
    moe.attn_key_weights(q, kc, table, starts(q_lens), ints(kv_lens), lse, w, causal=False)
    q[0] = 0
    want, tol = weights_reference(q, q_lens, kv_lens, kc, table, False, D ** -0.5, lse, torch.zeros_like(w))
    ref.check(w, want, tol, "weights")


@pytest.mark.parametrize("rows", [1, 150])
@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_scales(rows, scale):
    Hq, Hkv, D, page, q_lens, kv_lens = 12, 2, 128, 16, [rows, rows], [300, 200]
    kc, vc, table, _ = page_pool(kv_lens, page, Hkv, D, BF, 12)
    q = rand(gen_of(13), sum(q_lens), Hq, D)
    lse = torch.empty(sum(q_lens), Hq, device="cuda")
    moe.attn_prefill_paged(q, kc, torch.zeros_like(kc), table, starts(q_lens), ints(kv_lens), scale=scale, lse=lse)
    w = torch.zeros(2, Hkv, 300, device="cuda")
    moe.attn_key_weights(q, kc, table, starts(q_lens), ints(kv_lens), lse, w, scale=scale)
    want, tol = weights_reference(q, q_lens, kv_lens, kc, table, True, scale, lse, torch.zeros_like(w))
    ref.check(w, want, tol, "weights")
