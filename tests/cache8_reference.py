"""The paged cache in 8 bits from its definition in 64 bits: rounding to e4m3,
scales of 16 tokens and a head, and the keys and values that codes stand for."""
from __future__ import annotations

import torch

import attn_reference as ref

BLOCK = 16
F8 = torch.float8_e4m3fn


def round8(x):
    """The nearest e4m3 value (three bits after the leading one, steps of 2^-9 below 2^-6), ties to even, at most 448;
    NaN stays."""
    x = x.double()
    mag = x.abs().clamp(max=448.0)
    lead = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6).nan_to_num(1.0)))
    step = torch.exp2(lead - 3)
    return torch.where(x.isnan(), x, torch.sign(x) * (torch.round(mag / step) * step).clamp(max=448.0))


def scale_of(top: float) -> float:
    """The smallest 2^e, -24 <= e <= 7, with top <= 448 * 2^e (2^7 where there is none)."""
    for e in range(-24, 8):
        if top <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 7


def values(codes):
    return codes.view(torch.uint8).cpu().view(F8).double()


def rows(cache, scales, which, pages, n):
    """The first n rows [Hkv, n, D] (fp64, on the GPU) of a page list; which: 0 keys, 1 values."""
    got = cache.view(torch.uint8)[pages.long()].view(F8).double()
    s = scales[pages.long()][..., which].double()
    got = (got.unflatten(2, (-1, BLOCK)) * s[..., None, None]).flatten(2, 3)
    return got.permute(1, 0, 2, 3).reshape(got.shape[1], -1, got.shape[3])[:, :n]


def attend(q, k, v, scale, seen=None, parts=False):
    """attn_reference.attend over decoded keys and values (fp64) with what the kernels' arithmetic on codes adds:

    P, in f16, is formed with the exponent of its values' scale in it, so a weight below 2^-14 of the largest
    contribution rounds on a grid of 2^-24 of it: m keys, each off by at most 2^-25 2^max(s + e) 448, and the largest
    contribution's block holds a value above 224 2^e, so that this is at most m 2^-24 max |v|.  The exponents (|e| <=
    24) pass through three fp32 additions: a weight is off by 72 2^-24 more.  A row of bf16 queries is scaled by a power
    of two to f16, which rounds elements below 2^-28 of the largest to 2^-39 of it.

    parts (prefill): a row of queries, its largest brought to (224, 448], is a sum of e4m3 parts that is exact but for
    elements whose last bit lies below 2^-9 - bf16 below 2^-2, f16 below 2 - which are off by at most 2^-10: elements
    below 2^-9.8 (2^-6.8) of the largest by 2^-17.8 of it.  Values take the scale 2^top of their 128 keys, in f16: off by
    2^-25 2^top each, less than the m 2^-24 max |v| above, as the block with that scale holds a value above 224 2^top."""
    out, lse, tol_o, tol_l = ref.attend(q, k, v, scale, seen)
    m = k.shape[1]
    if m and q.shape[0]:
        vmax = v.nan_to_num(0.0, 0.0, 0.0).abs().amax()
        small = 2.0 ** -39 * q.double().abs().amax(-1) * k.nan_to_num(0.0).abs().sum(-1).amax() * abs(scale)
        if parts:
            top = q.double().abs().amax(-1, keepdim=True)
            fine = q.double().abs() < 2.0 ** (-9.8 if q.dtype == torch.bfloat16 else -6.8) * top     # [n, Hq, D]
            kmax = k.nan_to_num(0.0).abs().amax(1).repeat_interleave(q.shape[1] // k.shape[0], 0)    # [Hq, D]
            small = small + 2.0 ** -17.8 * top[..., 0] * (fine * kmax).sum(-1) * abs(scale)
        delta = 72 * 2.0 ** -24 + small                                     # [n, Hq]
        tol_o = tol_o + ((4 * delta + m * 2.0 ** -24) * vmax)[..., None]
        tol_l = torch.where(lse == -float("inf"), tol_l, tol_l + 2 * delta)
    return out, lse, tol_o, tol_l
