"""Attention operators from their definitions in 64 bits (plain torch, one
sequence and one head at a time), and the error bounds of the kernels'
arithmetic that the tests compare with."""
from __future__ import annotations

import math

import torch

# unit roundoff of the element types (round to nearest)
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# f16 rounds below 2^-14 on a grid of 2^-24; bf16's range is fp32's
SUB = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


def rope(x, weight, eps, cos, sin, rot, interleaved):
    """x [T, heads, D] fp64; cos, sin [T, rot/2]."""
    x = x.double()
    if weight is not None:
        x = x * weight.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = x.clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = cos[:, i].double()[:, None], sin[:, i].double()[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rope_bound(ref, dtype):
    # one rounding to the type, and fp32: the norm's sum of D <= 128 squares in
    # a tree (12 roundings, halved by the root), its root, quotient and two
    # products, and three roundings of the rotation, whose error is relative to
    # the pair's magnitude: 20 roundings cover them
    return U[dtype] * ref.abs() + 20 * 2.0 ** -24 * 1.5 * ref.abs().amax(-1, keepdim=True) + SUB[dtype]


def paged(cache, pages, n):
    """The first n rows [Hkv, n, D] of a page list."""
    k = cache[pages.long()]                       # [pages, Hkv, page_size, D]
    return k.permute(1, 0, 2, 3).reshape(k.shape[1], -1, k.shape[3])[:, :n]


def attend(q, k, v, scale, seen=None):
    """One sequence: q [n, Hq, D], k and v [Hkv, m, D], seen [n, m] bool or
    None.  Returns out, lse, and the bounds on their errors, all fp64.

    Bounds: a logit is an fp32 sum of D exact products (D roundings, relative
    to sum |q k|) and its scaling; p = exp of it is rounded to the type before
    it multiplies v (u, or f16's absolute grid, at least one p of a row is not
    below 1 before normalisation); the sum over m keys rounds at most m + 16
    times; the result rounds once.  A term p v is off by its factor's relative
    error, so the absolute error is that times sum p |v|."""
    dtype = q.dtype
    n, Hq, D = q.shape
    Hkv, m, _ = k.shape
    group = Hq // Hkv
    q, k, v = q.double(), k.double(), v.double()
    out = torch.zeros(n, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol_o = torch.zeros_like(out)
    tol_l = torch.zeros_like(lse)
    if m == 0 or n == 0:
        return out, lse, tol_o, tol_l
    for h in range(Hq):
        kk, vv = k[h // group], v[h // group]
        s = q[:, h] @ kk.T * scale
        mag = q[:, h].abs() @ kk.abs().T * abs(scale)
        if seen is not None:
            s = s.masked_fill(~seen, -math.inf)
            mag = mag.masked_fill(~seen, 0.0)
        top = s.amax(1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        e = torch.exp(s - top)
        total = e.sum(1, keepdim=True)
        p = e / torch.where(total == 0, torch.ones_like(total), total)
        vs = torch.where(torch.isfinite(vv), vv, torch.zeros_like(vv)) if seen is not None else vv
        out[:, h] = p @ vs
        lse[:, h] = (top + torch.log(total)).squeeze(1)
        delta = ((D + 4) * 2.0 ** -24 * mag.amax(1) + 2.0 ** -21)[:, None]
        summed = (m + 16) * 2.0 ** -24
        weight = p @ vs.abs()
        tol_o[:, h] = (U[dtype] * out[:, h].abs() + (U[dtype] + 4 * delta + 2 * summed + 2.0 ** -19) * weight
                       + SUB[dtype] * (2 * m * vs.abs().amax(0) + 1) + 1e-30)
        tol_l[:, h] = 2 * delta.squeeze(1) + summed + 2.0 ** -21 * (4 + lse[:, h].abs())
    empty = lse == -math.inf
    tol_l[empty] = 0.0
    return out, lse, tol_o, tol_l


def causal(n, m, device):
    """seen[i, j]: row i of n sees key j of m, the last row the last key."""
    return (torch.arange(m, device=device)[None, :] <= torch.arange(n, device=device)[:, None] + (m - n))


def check(got, ref, tol, what):
    got = got.double()
    both = torch.isinf(got) & torch.isinf(ref) & (got == ref)
    err = torch.where(both, torch.zeros_like(ref), (got - ref).abs())
    ok = err <= tol
    assert bool(ok.all()), (f"{what}: {int((~ok).sum())} of {ok.numel()} values off, worst "
                            f"{float((err / tol.clamp(min=1e-300))[~ok].max()):.3g} times the bound at "
                            f"{torch.nonzero(~ok)[0].tolist()}")
