"""GPU test of what attention and the MoE layer contribute to the rows that the
decoder-layer example serves, each taken before it is added to the residual
stream (of which it is a few percent) and compared with 64-bit torch on the
CPU; references with a mistake in them must be out of bounds."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -8            # unit roundoff of bf16

# Both branches, relative to a row's norm.  Attention: the normed input, q, k
# and v (a product's result each), the rotated q and k, P and the output are
# rounded to bf16.  An error of u of a random sign in each of a sum's terms is
# at most u of the sum's own size for values of random signs; logits are about
# N(0, 1), so that their error, of six roundings' root sum, is that of the
# weights: v and its input, P, the output and the logits' sqrt(6) u linearly are
# 6.5 u in the worst case, about 1.3 u in the mean square.  The MoE layer: gate
# and up, their product and the output, about as much.  Six of them bound a
# row's norm, in which hundreds of errors average.
BOUND = 6 * U

SHAPES = {
    "D64": dict(H=512, Hq=8, Hkv=2, D=64, E=8, top_k=2, I=256, pages=256),
    "D128": dict(H=1024, Hq=16, Hkv=2, D=128, E=8, top_k=8, I=256, page=32, pages=256),
}
SHARED, PROMPTS, STEPS = 64, [1, 24, 47, 70], 3


@pytest.fixture(scope="module", params=list(SHAPES))
def served(request):
    """The layer, its inputs on the CPU, and what its branches gave: one entry per call of finish()."""
    from expert_layer_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)

    class Recorder(m.DecoderLayer):
        calls = []

        def finish(self, x, attended):
            self.calls.append(dict(x=x, attended=attended))
            out = super().finish(x, attended)
            self.calls[-1]["out"] = out
            return out

        def experts(self, x):
            y = super().experts(x)
            self.calls[-1].update(normed=x, moe=y)
            return y
    layer = Recorder(seed=5, **SHAPES[request.param])
    layer.calls = []
    g = torch.Generator(device="cuda").manual_seed(6)

    def rows(n):
        return torch.randn(n, layer.H, generator=g, device="cuda").to(torch.bfloat16)
    system, prompts, steps = rows(SHARED), [rows(n) for n in PROMPTS], [rows(len(PROMPTS)) for _ in range(STEPS)]
    m.serve(layer, system, prompts, steps)
    torch.cuda.synchronize()
    return layer, system.cpu(), [p.cpu() for p in prompts], [s.cpu() for s in steps]


def attention(layer, rows, mistake=None):
    """[n, Hq, D] fp64 of these rows as one prompt; `mistake`: one planted in it."""
    x = rows.double()
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    Hq, Hkv, D, n = layer.Hq, layer.Hkv, layer.D, rows.shape[0]
    qkv = (x @ layer.w_qkv.cpu().double().T).view(n, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    position = torch.arange(n, dtype=torch.float64)
    if mistake == "positions start again":
        position = torch.where(position < SHARED, position, position - SHARED)
    angle = position[:, None] * 1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def turned(x):
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        if mistake == "not rotated":
            return x
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    q, k = turned(q), turned(k)
    seen = torch.ones(n, n, dtype=torch.bool).tril()
    own = torch.arange(n) >= SHARED
    if mistake == "no causal mask":
        seen[:] = True
    if mistake == "own keys dropped":
        seen &= ~(own[:, None] & own[None, :])
    if mistake == "prefix dropped":
        seen &= ~(own[:, None] & ~own[None, :])
    if mistake == "last key dropped":
        seen &= ~(own[:, None] & torch.eye(n, dtype=torch.bool))
    out = torch.empty(n, Hq, D, dtype=torch.float64)
    for h in range(Hq):
        kv = h * Hkv // Hq if mistake != "wrong heads" else h % Hkv
        s = (q[:, h] @ k[:, kv].T / math.sqrt(D)).masked_fill(~seen, -math.inf)
        out[:, h] = torch.softmax(s, 1) @ v[:, kv]
    return torch.zeros_like(out) if mistake == "nothing" else out


def error(got, want):
    """Largest error of a row over its norm."""
    d = (got.double().flatten(1) - want.flatten(1)).norm(dim=1) / want.flatten(1).norm(dim=1).clamp(min=1e-30)
    return float(d.max())


def by_request(layer, prompts, key):
    """Rows of each request in order: its prompt's, then one of every step."""
    parts = [c[key].cpu() for c in layer.calls]
    at = [sum(p.shape[0] for p in prompts[:i]) for i in range(len(prompts) + 1)]
    return [torch.cat([parts[1][at[r]:at[r + 1]]] + [s[r:r + 1] for s in parts[2:]]) for r in range(len(prompts))]


def test_attention_of_served_rows(served):
    layer, system, prompts, steps = served
    assert error(layer.calls[0]["attended"].cpu(), attention(layer, system)) <= BOUND
    for r, got in enumerate(by_request(layer, prompts, "attended")):
        rows = torch.cat([system, prompts[r]] + [s[r:r + 1] for s in steps])
        assert error(got, attention(layer, rows)[SHARED:]) <= BOUND, f"request {r}"


@pytest.mark.parametrize("mistake", ["nothing", "not rotated", "positions start again", "own keys dropped", "prefix dropped",
                                     "last key dropped", "no causal mask", "wrong heads"])
def test_attention_with_a_mistake_is_out_of_bounds(served, mistake):
    layer, system, prompts, steps = served
    for r, got in enumerate(by_request(layer, prompts, "attended")):
        rows = torch.cat([system, prompts[r]] + [s[r:r + 1] for s in steps])
        assert error(got, attention(layer, rows, mistake)[SHARED:]) > 2 * BOUND, f"request {r}"


def test_experts_of_served_rows(served):
    layer, checked, total = served[0], 0, 0
    gate, gu, down = (w.cpu().double() for w in (layer.gate_w, layer.w_gate_up, layer.w_down))
    for c in layer.calls:
        x, y = c["normed"].cpu().double(), c["moe"].cpu()
        logits = x @ gate.T
        top, at = logits.topk(layer.top_k, dim=1)
        weight = torch.softmax(top, 1)
        want = torch.zeros(x.shape[0], layer.H, dtype=torch.float64)
        for t in range(x.shape[0]):
            for w, e in zip(weight[t], at[t]):
                g, u = (gu[e] @ x[t]).chunk(2)
                want[t] += w * (down[e] @ (g * torch.sigmoid(g) * u))
        # rows whose last expert in and first one out nearly tie may take either
        sure = torch.ones(x.shape[0], dtype=torch.bool)
        if layer.top_k < logits.shape[1]:
            ordered = logits.sort(1, descending=True).values
            sure = ordered[:, layer.top_k - 1] - ordered[:, layer.top_k] > 1e-4
        assert error(y[sure], want[sure]) <= BOUND
        assert error(torch.zeros_like(y[sure]), want[sure]) > 2 * BOUND
        assert error(y[sure], want[sure].roll(1, 0)) > 2 * BOUND or int(sure.sum()) == 1
        checked, total = checked + int(sure.sum()), total + x.shape[0]
    assert checked > 0.95 * total


def test_served_rows_are_the_sum_of_their_parts(served):
    layer = served[0]
    for c in layer.calls:
        x = c["x"] + c["attended"].flatten(1) @ layer.w_o.T
        assert torch.equal(layer.norm(x), c["normed"])
        assert torch.equal(x + c["moe"], c["out"])
