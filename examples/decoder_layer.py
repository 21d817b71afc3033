#!/usr/bin/env python
"""One decoder layer served end to end: attention over the paged cache, then the MoE layer.

    python examples/decoder_layer.py [--requests 8] [--prompt 300] [--steps 4]

Requests share a system prompt.  The layer
  1. runs the shared prompt once (rope_append into its pages, attn_prefill_paged),
  2. runs every request's own prompt as a ragged batch that reads the shared pages (attn_prefill_paged),
  3. decodes token by token for the whole batch (rope_append, attn_decode with the shared prefix),
each followed by the output projection and the MoE layer (``forward``), and checks the served rows against
running the same tokens as one prompt (attn_prefill over packed rows).  Weights and inputs are random; the dense projections are torch products.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import expert_layer_gb300 as moe  # noqa: E402


class DecoderLayer:
    """Random weights of one layer and its paged cache."""

    def __init__(self, H=2048, Hq=32, Hkv=4, D=128, E=32, top_k=4, I=768, page=16, pages=2048, max_pos=8192, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, std=0.02):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)
        self.H, self.Hq, self.Hkv, self.D, self.page, self.top_k = H, Hq, Hkv, D, page, top_k
        self.w_qkv, self.w_o = w((Hq + 2 * Hkv) * D, H), w(H, Hq * D)
        self.gate_w, self.w_gate_up, self.w_down = w(E, H), w(E, 2 * I, H), w(E, H, I)
        self.q_norm, self.k_norm = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
        self.table = moe.rope_table(max_pos, D, base=1e6)
        self.k_cache = torch.empty(pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
        self.v_cache = torch.empty_like(self.k_cache)
        self.free = list(range(pages))

    def take_pages(self, tokens):
        n = (tokens + self.page - 1) // self.page
        if n > len(self.free):
            raise RuntimeError(f"the cache has {len(self.free)} free pages, {n} are needed")
        got, self.free = self.free[:n], self.free[n:]
        return got

    def slots(self, pages, start, count):
        """Cache slots of tokens start .. start + count - 1 of a page list."""
        return [pages[t // self.page] * self.page + t % self.page for t in range(start, start + count)]

    @staticmethod
    def norm(x):
        return (x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def queries(self, x, positions, slots):
        """Projection, head norms, rotation and the append to the cache: queries [T, Hq, D]."""
        T, Hq, Hkv, D = x.shape[0], self.Hq, self.Hkv, self.D
        qkv = self.norm(x) @ self.w_qkv.T
        self.k = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        self.v = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        return moe.rope_append(qkv[:, :Hq * D].view(T, Hq, D), self.k, self.v, self.table, ints(positions), ints(slots),
                               self.k_cache, self.v_cache, q_norm=self.q_norm, k_norm=self.k_norm)

    def experts(self, x):
        """The MoE layer on normed rows."""
        return moe.forward(x, self.gate_w, None, self.w_gate_up, self.w_down, self.top_k)

    def finish(self, x, attended):
        """Output projection and MoE layer, each added to its input."""
        x = x + attended.flatten(1) @ self.w_o.T
        return x + self.experts(self.norm(x))


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def table_of(lists):
    wide = max(1, max(len(p) for p in lists))
    return ints([p + [0] * (wide - len(p)) for p in lists])


def serve(layer, shared, prompts, steps):
    """shared [S, H], prompts: a list of [n_i, H], steps: a list of [B, H] (one new token of each request per step).
    Returns the layer's output rows: (shared, of the prompts, of each step)."""
    S, B = shared.shape[0], len(prompts)
    lens = [p.shape[0] for p in prompts]
    assert S % layer.page == 0, "the requests' page lists go on where the shared one ends"
    prefix = layer.take_pages(S)
    own = [layer.take_pages(n + len(steps)) for n in lens]

    # 1. the shared prompt, its keys read back from the pages they were just appended to
    q = layer.queries(shared, list(range(S)), layer.slots(prefix, 0, S))
    att = moe.attn_prefill_paged(q, layer.k_cache, layer.v_cache, table_of([prefix]), ints([0, S]), ints([S]))
    out_shared = layer.finish(shared, att)

    # 2. the requests' own prompts: keys are the shared pages, then their own
    x = torch.cat(prompts)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    q = layer.queries(x, [S + t for n in lens for t in range(n)],
                      [s for p, n in zip(own, lens) for s in layer.slots(p, 0, n)])
    att = moe.attn_prefill_paged(q, layer.k_cache, layer.v_cache, table_of([prefix + p for p in own]), ints(starts),
                                 ints([S + n for n in lens]))
    out_prompts = layer.finish(x, att)

    # 3. decode: the shared pages once for the batch, then each row's own
    own_table, prefix_table = table_of(own), ints(prefix)
    ws = moe.alloc_attn_workspace(B, B, layer.Hq, layer.Hkv, layer.D)
    outs = []
    for i, x in enumerate(steps):
        q = layer.queries(x, [S + n + i for n in lens], [layer.slots(p, n + i, 1)[0] for p, n in zip(own, lens)])
        att = moe.attn_decode(q, layer.k_cache, layer.v_cache, own_table, ints([n + i + 1 for n in lens]),
                              prefix_table, S, workspace=ws)
        if moe.read_status(ws) != 0:
            raise RuntimeError("device status reported an error")
        outs.append(layer.finish(x, att))
    return out_shared, out_prompts, outs


def as_one_prompt(layer, rows):
    """The layer's output for these rows as a single prompt, keys in packed rows (rotated copies from the cache)."""
    n = rows.shape[0]
    pages = layer.take_pages(n)
    q = layer.queries(rows, list(range(n)), layer.slots(pages, 0, n))
    ids = ints(pages).long()
    k, v = (c[ids].transpose(1, 2).reshape(-1, layer.Hkv, layer.D)[:n] for c in (layer.k_cache, layer.v_cache))
    return layer.finish(rows, moe.attn_prefill(q, k, v, ints([0, n]), ints([0, n])))


def run(requests=8, prompt=300, steps=4, shared=512, seed=0, **shape):
    """Serve a random batch; the largest difference of a served row from the same row of one whole prompt,
    over the largest value.  Rows that take the same experts both ways differ by bf16 roundings (6.5e-3 at the
    defaults); a row whose router logits nearly tie (one of 1388 there, 9e-4 apart) may take another expert and
    then differs by that expert's share (3.5e-2)."""
    layer = DecoderLayer(seed=seed, **shape)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)

    def rows(n):
        return torch.randn(n, layer.H, generator=g, device="cuda").to(torch.bfloat16)
    system = rows(shared)
    prompts = [rows(1 + (prompt * (i + 1)) // requests) for i in range(requests)]
    new = [rows(requests) for _ in range(steps)]
    _, out_prompts, outs = serve(layer, system, prompts, new)
    worst, at = 0.0, 0
    for r, p in enumerate(prompts):
        whole = as_one_prompt(layer, torch.cat([system, p] + [x[r:r + 1] for x in new]))[shared:].float()
        got = torch.cat([out_prompts[at:at + p.shape[0]]] + [x[r:r + 1] for x in outs]).float()
        worst = max(worst, float((got - whole).abs().max() / whole.abs().max()))
        at += p.shape[0]
    return worst


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--prompt", type=int, default=300, help="tokens of the longest prompt")
    p.add_argument("--steps", type=int, default=4)
    a = p.parse_args()
    worst = run(a.requests, a.prompt, a.steps)
    print(f"{a.requests} requests, {a.steps} decode steps: rows agree with whole prompts within {worst:.2e} of the "
          "largest value")


if __name__ == "__main__":
    main()
