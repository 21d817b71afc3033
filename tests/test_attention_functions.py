"""CPU tests of the attention functions as Python objects: the compiled ones
that take over at the first call have the same signatures and documentation."""
import subprocess
import sys

import pytest

from expert_layer_gb300 import _build

ROOT = _build.ROOT
SCRIPT = """
import inspect
import torch
import expert_layer_gb300 as moe
from expert_layer_gb300 import attention

NAMES = ["rope_append", "attn_prefill", "attn_prefill_paged", "attn_decode"]
def seen(module):
    return {n: (str(inspect.signature(getattr(module, n))), inspect.getdoc(getattr(module, n))) for n in NAMES}
before, early = seen(moe), moe.attn_decode
assert before == seen(attention) and all(len(d) > 100 for _, d in before.values())
q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
try:
    moe.attn_decode(q, q, q, q, q)
    raise SystemExit("not refused")
except moe.MoEError:
    pass
assert moe.attn_decode is not early, "the compiled functions did not take over"
assert seen(moe) == before and seen(attention) == before
for n in NAMES:
    # parameters may be named, in any order, and defaults left out; refusals do not change with the way
    names = list(inspect.signature(getattr(moe, n)).parameters)
    texts = set()
    for call in (lambda f: f(*[q] * len(names)), lambda f: f(**{p: q for p in reversed(names)}),
                 lambda f: f(q, **{p: q for p in names[1:]})):
        for f in (getattr(moe, n), next(w for w in attention._FUNCTIONS if w.__name__ == n)):
            try:
                call(f)
            except moe.MoEError as e:
                texts.add(str(e))
    assert len(texts) == 1, texts
print("same")
"""


def test_signatures_and_documentation_stay():
    _build.build()
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_bind_checks_the_definitions():
    import expert_layer_gb300 as moe
    from expert_layer_gb300 import attention
    native = attention._load()
    with pytest.raises(TypeError):
        native.bind(moe.MoEError, 0, 0, 0, 0, 0, 0, *[(("q",), (), "")] * 4)
